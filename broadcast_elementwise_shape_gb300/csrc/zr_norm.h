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
  // The ring: stages (2 or 3), 16-byte units per row and input, dynamic shared
  // memory in all.  raw: element-wise rows of neighbouring elements; out_pairs: rows of a
  // 2-byte output start at 4-byte boundaries.
  uint32_t stages, slot, smem, raw, out_pairs;
};

constexpr int kNormThreads = 256;
// CTAs per SM that the kernels' registers allow without spills, by columns per
// lane, forward and backward alike.
ZR_CX int norm_occ(int cols) { return cols > 16 ? 2 : (cols > 8 ? 3 : 4); }
constexpr int kNormSmemMax = 224 * 1024; // dynamic shared memory of all CTAs of an SM
constexpr uint32_t kNormLongThreads = 1024;
constexpr uint32_t kNormSumCols = 32;    // k_norm_sums: columns per CTA

// Vectors (elements) per lane that a plan may use, per access width, close
// enough that lanes of the larger groups idle for a quarter of a row at most.
// One list for the planner and the launchers (ZR_NORM_CASE(G, NI)).
#define ZR_NORM_CASES(VEC_)                                                        \
  if constexpr (VEC_ == 1) {                                                       \
    ZR_NORM_CASE(8, 4) ZR_NORM_CASE(8, 8) ZR_NORM_CASE(32, 4) ZR_NORM_CASE(32, 8)   \
    ZR_NORM_CASE(32, 12) ZR_NORM_CASE(32, 16) ZR_NORM_CASE(64, 12)                 \
    ZR_NORM_CASE(64, 16) ZR_NORM_CASE(128, 12) ZR_NORM_CASE(128, 16)               \
    ZR_NORM_CASE(256, 12) ZR_NORM_CASE(256, 16) ZR_NORM_CASE(256, 24) ZR_NORM_CASE(256, 32) \
  } else if constexpr (VEC_ == 4) {                                                \
    ZR_NORM_CASE(8, 1) ZR_NORM_CASE(8, 2)                                          \
    ZR_NORM_CASE(32, 1) ZR_NORM_CASE(32, 2) ZR_NORM_CASE(32, 4) ZR_NORM_CASE(32, 6) \
    ZR_NORM_CASE(32, 8) ZR_NORM_CASE(64, 4) ZR_NORM_CASE(64, 6) ZR_NORM_CASE(64, 8) \
    ZR_NORM_CASE(128, 4) ZR_NORM_CASE(128, 6) ZR_NORM_CASE(128, 8)                 \
    ZR_NORM_CASE(256, 1) ZR_NORM_CASE(256, 2) ZR_NORM_CASE(256, 4)                 \
    ZR_NORM_CASE(256, 6) ZR_NORM_CASE(256, 8)                                      \
  } else {                                                                         \
    ZR_NORM_CASE(8, 1) ZR_NORM_CASE(8, 2)                                          \
    ZR_NORM_CASE(32, 1) ZR_NORM_CASE(32, 2) ZR_NORM_CASE(32, 3) ZR_NORM_CASE(32, 4) \
    ZR_NORM_CASE(64, 2) ZR_NORM_CASE(64, 3) ZR_NORM_CASE(64, 4)                    \
    ZR_NORM_CASE(128, 2) ZR_NORM_CASE(128, 3) ZR_NORM_CASE(128, 4)                 \
    ZR_NORM_CASE(256, 1) ZR_NORM_CASE(256, 2) ZR_NORM_CASE(256, 3) ZR_NORM_CASE(256, 4) \
  }

// vec: elements per access, 16 bytes' worth or 1.
cudaError_t launch_norm_fwd(const NormPlan& p, int es, int vec, cudaStream_t s);
// The column sums' partials (when p.partial) come from the same pass, or for
// long rows from k_norm_sums, launched first.
cudaError_t launch_norm_bwd(const NormPlan& p, int es, int vec, cudaStream_t s);

}  // namespace zr
