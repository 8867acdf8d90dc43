// zr_norm.h — layer norm's kernel plan (passed by value) and its launchers.
#pragma once

#include <cuda_runtime.h>

#include "zr_internal.h"

namespace zr {

// Rows of `dim` elements.  Slot 0 is x (forward) or grad_out (backward),
// slot 1 x (backward), slot 3 the output.
struct NormPlan {
  const void* in[2];
  void* out;                 // y or grad_x; null: not written (backward)
  const void* gamma;         // null: 1
  const void* beta;          // null: 0 (forward)
  float* mean;               // forward: written unless null
  float* rstd;
  const float* mean_in;      // backward: read
  const float* rstd_in;
  float* partial;            // backward: [n_cta][n_part * dim] column sums, or null
  Decomp rows;               // row -> offsets of slots 0, 1, 3
  int64_t inner_stride[kMaxOperands];
  int64_t gamma_stride, beta_stride;
  uint32_t nrow, dim;
  float eps, inv_dim;
  uint32_t want_gamma, want_beta;  // backward: which column sums are kept
  uint32_t affine_vec;       // gamma and beta (where given) take vector loads
  // Row-resident kernels: `group` lanes per row, ni vectors per lane.
  // group == 0: rows longer than a block holds in registers.
  uint32_t group, ni;
  uint32_t n_cta;
  uint32_t stages, smem;     // ring stages (2 or 3), dynamic shared memory
};

constexpr int kNormThreads = 256;
// k_norm_fwd likewise.
ZR_CX int norm_fwd_occ(int cols, int vec) {
  return vec == 1 ? (cols > 16 ? 3 : 4) : (cols > 16 ? 2 : (cols > 8 ? 3 : 4));
}
// k_norm_bwd: CTAs per SM its registers allow without spills, by columns per
// lane (element-wise access keeps the row in registers too).
ZR_CX int norm_bwd_occ(int cols, int vec) {
  return vec == 1 ? (cols > 16 ? 1 : (cols > 8 ? 2 : (cols > 4 ? 3 : 4)))
                  : (cols > 16 ? 2 : (cols > 8 ? 3 : 4));
}
constexpr int kNormSmemMax = 224 * 1024; // dynamic shared memory of all CTAs of an SM
constexpr uint32_t kNormMaxCols = 32;    // columns per lane held in registers
constexpr uint32_t kNormLongThreads = 1024;
constexpr uint32_t kNormSumCols = 32;    // k_norm_sums: columns per CTA

// Vectors per lane that a plan may use, per access width: enough steps that no
// lane of a full row group holds more than 1.5 times the columns it needs.
// One list for the planner and the launchers (ZR_NORM_CASE(G, NI)).
#define ZR_NORM_CASES(VEC_)                                                       \
  if constexpr (VEC_ == 1) {                                                      \
    ZR_NORM_CASE(8, 4) ZR_NORM_CASE(8, 8) ZR_NORM_CASE(32, 4) ZR_NORM_CASE(32, 8)  \
    ZR_NORM_CASE(256, 2) ZR_NORM_CASE(256, 4) ZR_NORM_CASE(256, 8)                \
    ZR_NORM_CASE(256, 16) ZR_NORM_CASE(256, 32)                                   \
  } else if constexpr (VEC_ == 4) {                                               \
    ZR_NORM_CASE(8, 1) ZR_NORM_CASE(8, 2)                                         \
    ZR_NORM_CASE(32, 1) ZR_NORM_CASE(32, 2) ZR_NORM_CASE(32, 4) ZR_NORM_CASE(32, 6) \
    ZR_NORM_CASE(32, 8) ZR_NORM_CASE(256, 2) ZR_NORM_CASE(256, 4) ZR_NORM_CASE(256, 8) \
  } else {                                                                        \
    ZR_NORM_CASE(8, 1) ZR_NORM_CASE(8, 2)                                         \
    ZR_NORM_CASE(32, 1) ZR_NORM_CASE(32, 2) ZR_NORM_CASE(32, 3) ZR_NORM_CASE(32, 4) \
    ZR_NORM_CASE(256, 1) ZR_NORM_CASE(256, 2) ZR_NORM_CASE(256, 4)                \
  }

// vec: elements per access, 16 bytes' worth or 1.
cudaError_t launch_norm_fwd(const NormPlan& p, int es, int vec, cudaStream_t s);
// The column sums' partials (when p.partial) come from the same pass, or for
// long rows from k_norm_sums, launched first.
cudaError_t launch_norm_bwd(const NormPlan& p, int es, int vec, cudaStream_t s);

}  // namespace zr
