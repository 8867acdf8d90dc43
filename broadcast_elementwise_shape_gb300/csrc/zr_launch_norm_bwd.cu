// zr_launch_norm_bwd.cu — layer norm backward launches.
#include "zr_norm.cuh"

namespace zr {
namespace {

template <typename E, int VEC, int G, int NI>
cudaError_t go(const NormPlan& p, cudaStream_t s) {
  auto* k = k_norm_bwd<E, VEC, G, NI>;
  if (p.smem > 40 * 1024) {  // with the static shared memory, under 48 KB otherwise
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), kNormSmemMax);
    if (e != cudaSuccess) return e;
  }
  return launch_k(k, p.n_cta, kNormThreads, p.smem, s, p);
}

template <typename E, int VEC>
cudaError_t pick(const NormPlan& p, cudaStream_t s) {
  if (p.group == 0) {
    if (p.partial) {
      const dim3 grid((p.dim + kNormSumCols - 1) / kNormSumCols, p.n_cta);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = grid;
      cfg.blockDim = dim3(kNormThreads);
      cfg.stream = s;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      const cudaError_t e = cudaLaunchKernelEx(&cfg, k_norm_sums<E>, p);
      if (e != cudaSuccess) return e;
    }
    if (!p.out) return cudaSuccess;
    return launch_k(k_norm_bwd_long<E, VEC>, p.nrow, kNormLongThreads, 0, s, p);
  }
#define ZR_NORM_CASE(G_, NI_) \
  if (p.group == G_ && p.ni == NI_) return go<E, VEC, G_, NI_>(p, s);
  ZR_NORM_CASES(VEC)
#undef ZR_NORM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_bwd(const NormPlan& p, int es, int vec, cudaStream_t s) {
  if (!p.in[0] || !p.in[1] || !p.mean_in || !p.rstd_in) return cudaErrorInvalidValue;
  if (es == 4) return vec == 4 ? pick<float, 4>(p, s) : pick<float, 1>(p, s);
  return vec == 8 ? pick<__nv_bfloat16, 8>(p, s) : pick<__nv_bfloat16, 1>(p, s);
}

}  // namespace zr
