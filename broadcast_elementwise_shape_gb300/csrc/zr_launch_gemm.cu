// zr_launch_gemm.cu — launches of the tensor-core product.
#include "zr_gemm.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

template <int EPI, int CG, bool SUM>
cudaError_t go(const GemmPlan& p, unsigned grid, cudaStream_t s) {
  auto* k = k_gemm<EPI, CG, SUM>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), int(GemmCfg<CG>::kSmem));
  if (e != cudaSuccess) return e;
  if (CG == 1) return launch_k(k, grid, kGemmThreads, GemmCfg<CG>::kSmem, s, p);
  return launch_k_cluster(k, grid, kGemmThreads, GemmCfg<CG>::kSmem, s, CG, p);
}

template <int EPI>
cudaError_t pick(int cg, bool sum, const GemmPlan& p, unsigned grid, cudaStream_t s) {
  if (cg == 1) return sum ? go<EPI, 1, true>(p, grid, s) : go<EPI, 1, false>(p, grid, s);
  return sum ? go<EPI, 2, true>(p, grid, s) : go<EPI, 2, false>(p, grid, s);
}

}  // namespace

cudaError_t launch_gemm(int epi, int cg, bool sum, const GemmPlan& p, unsigned grid,
                        cudaStream_t s) {
  if (grid == 0 || (cg != 1 && cg != 2) || grid % unsigned(cg) != 0) return cudaErrorInvalidValue;
  for (uint32_t i = 0; i < p.n_prob; ++i)
    if (p.pr[i].chunk == 0 || (!sum && p.pr[i].chunk < p.pr[i].n_kb)) return cudaErrorInvalidValue;
  switch (epi) {
    case kEpiLse: return pick<kEpiLse>(cg, sum, p, grid, s);
    case kEpiGrad: return pick<kEpiGrad>(cg, sum, p, grid, s);
    case kEpiOut: return pick<kEpiOut>(cg, sum, p, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace zr
