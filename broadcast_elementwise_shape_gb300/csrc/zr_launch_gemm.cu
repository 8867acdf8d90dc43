// zr_launch_gemm.cu — launches of the tensor-core product.
#include "zr_gemm.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

template <int EPI, int CG>
cudaError_t go(const GemmPlan& p, unsigned grid, cudaStream_t s) {
  auto* k = k_gemm<EPI, CG>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), int(GemmCfg<CG>::kSmem));
  if (e != cudaSuccess) return e;
  if (CG == 1) return launch_k(k, grid, kGemmThreads, GemmCfg<CG>::kSmem, s, p);
  return launch_k_cluster(k, grid, kGemmThreads, GemmCfg<CG>::kSmem, s, CG, p);
}

}  // namespace

cudaError_t launch_gemm(int epi, int cg, const GemmPlan& p, unsigned grid, cudaStream_t s) {
  if (grid == 0 || (cg != 1 && cg != 2) || grid % unsigned(cg) != 0) return cudaErrorInvalidValue;
  switch (epi * 2 + cg - 1) {
    case kEpiLse * 2: return go<kEpiLse, 1>(p, grid, s);
    case kEpiLse * 2 + 1: return go<kEpiLse, 2>(p, grid, s);
    case kEpiGrad * 2: return go<kEpiGrad, 1>(p, grid, s);
    case kEpiGrad * 2 + 1: return go<kEpiGrad, 2>(p, grid, s);
    case kEpiOut * 2: return go<kEpiOut, 1>(p, grid, s);
    case kEpiOut * 2 + 1: return go<kEpiOut, 2>(p, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace zr
