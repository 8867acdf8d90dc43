// zr_launch_norm_fwd.cu — layer norm forward launches.
#include "zr_norm.cuh"

namespace zr {
namespace {

template <typename E, int VEC, int G, int NI>
cudaError_t go(const NormPlan& p, cudaStream_t s) {
  auto* k = k_norm_fwd<E, VEC, G, NI>;
  if (p.smem > 40 * 1024) {  // with the static shared memory, under 48 KB otherwise
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), kNormSmemMax);
    if (e != cudaSuccess) return e;
  }
  return launch_k(k, p.n_cta, kNormThreads, p.smem, s, p);
}

template <typename E, int VEC>
cudaError_t pick(const NormPlan& p, cudaStream_t s) {
  if (p.group == 0) return launch_k(k_norm_fwd_long<E, VEC>, p.n_cta, kNormLongThreads, 0, s, p);
#define ZR_NORM_CASE(G_, NI_) \
  if (p.group == G_ && p.ni == NI_) return go<E, VEC, G_, NI_>(p, s);
  ZR_NORM_CASES(VEC)
#undef ZR_NORM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormPlan& p, int es, int vec, cudaStream_t s) {
  if (!p.in[0] || !p.out) return cudaErrorInvalidValue;
  if (es == 4) return vec == 4 ? pick<float, 4>(p, s) : pick<float, 1>(p, s);
  return vec == 8 ? pick<__nv_bfloat16, 8>(p, s) : pick<__nv_bfloat16, 1>(p, s);
}

}  // namespace zr
