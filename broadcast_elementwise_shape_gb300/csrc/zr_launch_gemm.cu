// zr_launch_gemm.cu — launches of the tensor-core product.
#include "zr_gemm.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

template <int EPI, int CG, bool SUM, int PARTS>
cudaError_t go(const GemmPlan& p, unsigned grid, cudaStream_t s) {
  auto* k = k_gemm<EPI, CG, SUM, PARTS>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), int(GemmCfg<EPI, CG, PARTS>::kSmem));
  if (e != cudaSuccess) return e;
  if (CG == 1) return launch_k(k, grid, kGemmThreads, GemmCfg<EPI, CG, PARTS>::kSmem, s, p);
  return launch_k_cluster(k, grid, kGemmThreads, GemmCfg<EPI, CG, PARTS>::kSmem, s, CG, p);
}

template <int EPI, int CG>
cudaError_t pick(bool sum, const GemmPlan& p, unsigned grid, cudaStream_t s) {
  if (p.parts == 3) return go<EPI, CG, true, 3>(p, grid, s);
  if constexpr (EPI != kEpiLse && CG == 1)  // G in two parts is for up to 128 rows
    if (p.parts == 2) return sum ? go<EPI, CG, true, 2>(p, grid, s) : go<EPI, CG, false, 2>(p, grid, s);
  return sum ? go<EPI, CG, true, 1>(p, grid, s) : go<EPI, CG, false, 1>(p, grid, s);
}

}  // namespace

cudaError_t launch_gemm(int epi, int cg, bool sum, const GemmPlan& p, unsigned grid,
                        cudaStream_t s) {
  if (grid == 0 || (cg != 1 && cg != 2) || grid % unsigned(cg) != 0) return cudaErrorInvalidValue;
  for (uint32_t i = 0; i < p.n_prob; ++i)
    if (p.pr[i].chunk == 0 || (!sum && p.pr[i].chunk < p.pr[i].kb_slice)) return cudaErrorInvalidValue;
  if (p.parts < 1 || p.parts > 3 || (p.parts == 3 && !sum) || (p.parts == 2 && (epi == kEpiLse || cg != 1)))
    return cudaErrorInvalidValue;
  const uint32_t widest = p.parts == 3 && cg == 1 ? 128 : 256;
  for (uint32_t i = 0; i < p.n_prob; ++i)
    if (p.pr[i].tn > widest) return cudaErrorInvalidValue;
  const bool two = cg == 2;
  switch (epi) {
    case kEpiLse: return two ? pick<kEpiLse, 2>(sum, p, grid, s) : pick<kEpiLse, 1>(sum, p, grid, s);
    case kEpiGrad: return two ? pick<kEpiGrad, 2>(sum, p, grid, s) : pick<kEpiGrad, 1>(sum, p, grid, s);
    case kEpiOut: return two ? pick<kEpiOut, 2>(sum, p, grid, s) : pick<kEpiOut, 1>(sum, p, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace zr
