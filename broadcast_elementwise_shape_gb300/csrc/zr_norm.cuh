// zr_norm.cuh — layer norm kernels (sm_103a).
//
// Forward, per row of D elements: mu = sum(x) / D, v = sum((x - mu)^2) / D,
// rstd = 1 / sqrt(v + eps), y = (x - mu) * rstd * gamma + beta.
// Backward, with xh = (x - mu) * rstd and q = g * gamma:
//   grad_x = rstd * (q - sum(q) / D - xh * sum(q * xh) / D),
//   grad_gamma = sum over rows of g * xh,  grad_beta = sum over rows of g.
// All arithmetic and every sum is binary32; outputs are rounded once.
//
// Both passes are bound by HBM: the forward must read x and write y, the
// backward read g and x and write grad_x.  So a row is read once and stays in
// registers (the variance is the two-pass one, from the differences, at no
// cost in traffic): G lanes hold a row of up to 32 columns each.  G = 8 for
// very short rows, a warp up to 1024 columns, a block of 256 up to 8192.
// Longer rows loop over the row, whose re-reads come from L1 and L2.
//
// In the backward a lane's columns are the same for every row it meets, so
// the two column sums build up in its registers over a persistent grid's
// rows; each block adds its row groups in a fixed order and writes one
// partial row, and the library's second pass adds the partials in order.  No
// atomics: the order is a function of the shape.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zr_kernels.cuh"
#include "zr_norm.h"

namespace zr {

template <typename E>
__device__ __forceinline__ float norm_ld(const E* p) {
  if constexpr (sizeof(E) == 2) return __bfloat162float(*p);
  else return *p;
}

// VEC elements from p (16 bytes when VEC > 1) as floats.
template <typename E, int VEC>
__device__ __forceinline__ void norm_load(const E* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = norm_ld(p);
  } else if constexpr (sizeof(E) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <typename E, int VEC>
__device__ __forceinline__ void norm_store(E* p, const float* v) {
  if constexpr (VEC == 1) {
    st1(p, v[0]);
  } else if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// gamma or beta at columns c .. c + VEC - 1 (`none` where it is not given).
template <typename E, int VEC>
__device__ __forceinline__ void norm_affine(const void* base, int64_t stride, uint32_t vec_ok,
                                            uint32_t c, float none, float* v) {
  if (base == nullptr) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = none;
    return;
  }
  const E* p = static_cast<const E*>(base);
  if (VEC > 1 && vec_ok) {
    norm_load<E, VEC>(p + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = norm_ld(p + int64_t(c + j) * stride);
  }
}

__device__ __forceinline__ void norm_row(const Decomp& dc, uint32_t row, int64_t* off) {
  if (dc.n <= 1) {
#pragma unroll
    for (int k = 0; k < kMaxOperands; ++k) off[k] = int64_t(row) * dc.stride[k][0];
  } else {
    decomp_offsets(dc, row, off);
  }
}

// Sum over the G lanes of a row group.  G <= 32: butterflies, every lane gets
// the same bits.  G = a block: warps by butterfly, then the warps' sums in
// order from s (one float per warp, not reused before the next barrier).
template <int G>
__device__ __forceinline__ float norm_sum(float v, float* s) {
#pragma unroll
  for (int m = (G < 32 ? G : 32) / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < G / 32; ++w) v += s[w];
  }
  return v;
}

template <typename E, int VEC, int G, int NI>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  __shared__ float s_sum[2][32];
  const uint32_t lane = threadIdx.x % G;
  const uint32_t row = blockIdx.x * (kNormThreads / G) + threadIdx.x / G;
  const bool live = row < p.nrow;  // whole row groups; a block's rows all live when G is a block
  int64_t off[kMaxOperands];
  norm_row(p.rows, live ? row : 0, off);
  const E* x = static_cast<const E*>(p.in[0]) + off[0];
  const int64_t xs = VEC > 1 ? 1 : p.inner_stride[0];
  pdl_wait();
  float v[NI][VEC];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t c = (i * G + lane) * VEC;
    if (live && c < p.dim) {
      norm_load<E, VEC>(x + int64_t(c) * xs, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += v[i][j];
  const float mean = __fmul_rn(norm_sum<G>(sum, s_sum[0]), p.inv_dim);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t c = (i * G + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      v[i][j] -= mean;
      if (c < p.dim) sq = __fmaf_rn(v[i][j], v[i][j], sq);
    }
  }
  const float var = __fmul_rn(norm_sum<G>(sq, s_sum[1]), p.inv_dim);
  const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
  if (!live) return;
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  E* y = static_cast<E*>(p.out) + off[kSlotOut];
  const int64_t ys = VEC > 1 ? 1 : p.inner_stride[kSlotOut];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t c = (i * G + lane) * VEC;
    if (c < p.dim) {
      float ga[VEC], be[VEC], o[VEC];
      norm_affine<E, VEC>(p.gamma, p.gamma_stride, p.affine_vec, c, 1.f, ga);
      norm_affine<E, VEC>(p.beta, p.beta_stride, p.affine_vec, c, 0.f, be);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = __fmaf_rn(v[i][j] * rstd, ga[j], be[j]);
      norm_store<E, VEC>(y + int64_t(c) * ys, o);
    }
  }
}

// Rows too long for a block's registers: one block per row, three walks over
// the row (sum, squared differences, output); the second and third read what
// the first brought into L1 and L2.
template <typename E, int VEC>
__global__ void __launch_bounds__(kNormLongThreads)
k_norm_fwd_long(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  __shared__ float s_sum[2][32];
  constexpr int G = kNormLongThreads;
  const uint32_t row = blockIdx.x;
  int64_t off[kMaxOperands];
  norm_row(p.rows, row, off);
  const E* x = static_cast<const E*>(p.in[0]) + off[0];
  const int64_t xs = VEC > 1 ? 1 : p.inner_stride[0];
  pdl_wait();
  float sum = 0.f;
  for (uint64_t c = threadIdx.x * VEC; c < p.dim; c += G * VEC) {
    float v[VEC];
    norm_load<E, VEC>(x + int64_t(c) * xs, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += v[j];
  }
  const float mean = __fmul_rn(norm_sum<G>(sum, s_sum[0]), p.inv_dim);
  float sq = 0.f;
  for (uint64_t c = threadIdx.x * VEC; c < p.dim; c += G * VEC) {
    float v[VEC];
    norm_load<E, VEC>(x + int64_t(c) * xs, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float d = v[j] - mean;
      sq = __fmaf_rn(d, d, sq);
    }
  }
  const float var = __fmul_rn(norm_sum<G>(sq, s_sum[1]), p.inv_dim);
  const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  E* y = static_cast<E*>(p.out) + off[kSlotOut];
  const int64_t ys = VEC > 1 ? 1 : p.inner_stride[kSlotOut];
  for (uint64_t c = threadIdx.x * VEC; c < p.dim; c += G * VEC) {
    float v[VEC], ga[VEC], be[VEC];
    norm_load<E, VEC>(x + int64_t(c) * xs, v);
    norm_affine<E, VEC>(p.gamma, p.gamma_stride, p.affine_vec, uint32_t(c), 1.f, ga);
    norm_affine<E, VEC>(p.beta, p.beta_stride, p.affine_vec, uint32_t(c), 0.f, be);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __fmaf_rn((v[j] - mean) * rstd, ga[j], be[j]);
    norm_store<E, VEC>(y + int64_t(c) * ys, v);
  }
}

// ------------------------------------------------------------------ backward

// The 16 bytes of VEC elements at `raw` as floats.
template <typename E, int VEC>
__device__ __forceinline__ void norm_unpack(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void norm_cp16(uint4* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
}

// A row group's lanes keep the two column sums of their columns in registers
// for all the rows the block meets.  What bounds the pass is the bytes in
// flight: with 16-byte vectors each lane copies the vectors it will read
// itself into its own slots of a shared-memory ring, p.stages - 1 rows ahead
// (cp.async: no registers, and no barrier since no lane reads another's), and
// reads them twice from there, once for the row's two means and the column
// sums, once for grad_x.  Keeping the row in registers instead took 222 of
// them and left 8 warps per SM: [65536, 1024] bf16 137 us against 78.
template <typename E, int VEC, int G, int NI>
__global__ void __launch_bounds__(kNormThreads, norm_bwd_occ(NI * VEC, VEC))
k_norm_bwd(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  constexpr int T = kNormThreads;
  constexpr int RPB = T / G;           // rows per block per step
  constexpr int W = G * NI * VEC;      // columns the lanes cover
  extern __shared__ uint4 s_ring[];    // [stage][row group][g, x][NI * G]; then column sums
  __shared__ float s_sum[2][2][32];
  const uint32_t lane = threadIdx.x % G, grp = threadIdx.x / G;
  const int64_t gs = VEC > 1 ? 1 : p.inner_stride[0];
  const int64_t xs = VEC > 1 ? 1 : p.inner_stride[1];
  const int64_t os = VEC > 1 ? 1 : p.inner_stride[kSlotOut];
  float acc_g[NI][VEC], acc_b[NI][VEC];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc_g[i][j] = acc_b[i][j] = 0.f;
  const uint64_t step = uint64_t(gridDim.x) * RPB;
  const uint64_t first = uint64_t(blockIdx.x) * RPB + grp;
  const uint32_t S = p.stages;
  auto slot = [&](uint32_t stage, int a) {
    return s_ring + ((uint64_t(stage) * RPB + grp) * 2 + a) * (NI * G) + lane;
  };
  auto fetch = [&](uint32_t stage, uint64_t row) {
    if constexpr (VEC > 1) {
      if (row < p.nrow) {
        int64_t off[kMaxOperands];
        norm_row(p.rows, uint32_t(row), off);
        const E* g = static_cast<const E*>(p.in[0]) + off[0];
        const E* x = static_cast<const E*>(p.in[1]) + off[1];
        uint4* sg = slot(stage, 0);
        uint4* sx = slot(stage, 1);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t c = (i * G + lane) * VEC;
          if (c < p.dim) {
            norm_cp16(sg + i * G, g + c);
            norm_cp16(sx + i * G, x + c);
          }
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
  };
  pdl_wait();
  if constexpr (VEC > 1)
    for (uint32_t k = 0; k + 1 < S; ++k) fetch(k, first + k * step);
  float mean = first < p.nrow ? p.mean_in[first] : 0.f;
  float rstd = first < p.nrow ? p.rstd_in[first] : 0.f;
  float gam[NI][VEC];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t c = (i * G + lane) * VEC;
    if (c < p.dim) {
      norm_affine<E, VEC>(p.gamma, p.gamma_stride, p.affine_vec, c, 1.f, gam[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) gam[i][j] = 0.f;
    }
  }
  uint32_t flip = 0, stage = 0, ahead = S - 1;
  for (uint64_t r0 = uint64_t(blockIdx.x) * RPB; r0 < p.nrow; r0 += step) {
    const uint64_t row = r0 + grp;
    const bool live = row < p.nrow;
    // The next row's statistics, and the vectors of the row S - 1 steps on.
    const float mean_next = row + step < p.nrow ? p.mean_in[row + step] : 0.f;
    const float rstd_next = row + step < p.nrow ? p.rstd_in[row + step] : 0.f;
    int64_t off[kMaxOperands];
    norm_row(p.rows, live ? uint32_t(row) : 0, off);
    if constexpr (VEC > 1) {
      fetch(ahead, row + (S - 1) * step);
      if (S == 3) asm volatile("cp.async.wait_group 2;\n" ::: "memory");
      else asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    }
    auto load = [&](int i, uint32_t c, float* gv, float* xv) {
      if constexpr (VEC > 1) {
        norm_unpack<E, VEC>(slot(stage, 0)[i * G], gv);
        norm_unpack<E, VEC>(slot(stage, 1)[i * G], xv);
      } else {
        gv[0] = norm_ld(static_cast<const E*>(p.in[0]) + off[0] + int64_t(c) * gs);
        xv[0] = norm_ld(static_cast<const E*>(p.in[1]) + off[1] + int64_t(c) * xs);
      }
    };
    // One access's values stay in registers between the two walks.
    float gk[VEC > 1 ? 1 : NI], xk[VEC > 1 ? 1 : NI];
    if constexpr (VEC == 1) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t c = i * G + lane;
        gk[i] = 0.f;
        xk[i] = mean;
        if (live && c < p.dim) load(i, c, &gk[i], &xk[i]);
      }
    }
    float sq = 0.f, sqx = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t c = (i * G + lane) * VEC;
      if (live && c < p.dim) {
        float gv[VEC], xv[VEC];
        if constexpr (VEC > 1) load(i, c, gv, xv);
        else { gv[0] = gk[i]; xv[0] = xk[i]; }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (xv[j] - mean) * rstd;
          acc_b[i][j] += gv[j];
          acc_g[i][j] = __fmaf_rn(gv[j], xh, acc_g[i][j]);
          const float q = gv[j] * gam[i][j];
          sq += q;
          sqx = __fmaf_rn(q, xh, sqx);
        }
      }
    }
    if (p.out) {
      const float m1 = __fmul_rn(norm_sum<G>(sq, s_sum[flip][0]), p.inv_dim);
      const float m2 = __fmul_rn(norm_sum<G>(sqx, s_sum[flip][1]), p.inv_dim);
      flip ^= 1;  // a block's next row writes the other pair: one barrier lies between
      E* o = static_cast<E*>(p.out) + off[kSlotOut];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t c = (i * G + lane) * VEC;
        if (live && c < p.dim) {
          float gv[VEC], xv[VEC];
          if constexpr (VEC > 1) load(i, c, gv, xv);
          else { gv[0] = gk[i]; xv[0] = xk[i]; }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float xh = (xv[j] - mean) * rstd;
            xv[j] = rstd * __fmaf_rn(-xh, m2, gv[j] * gam[i][j] - m1);
          }
          norm_store<E, VEC>(o + int64_t(c) * os, xv);
        }
      }
    }
    mean = mean_next;
    rstd = rstd_next;
    if (++stage == S) stage = 0;
    if (++ahead == S) ahead = 0;
  }
  if (!p.partial) return;
  const uint32_t nw = p.want_gamma + p.want_beta;
  float* part = p.partial + uint64_t(blockIdx.x) * nw * p.dim;
  float* s_col = reinterpret_cast<float*>(s_ring);  // [W]: the ring's copies are all in
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float(&acc)[NI][VEC] = k == 0 ? acc_g : acc_b;
    if (!(k == 0 ? p.want_gamma : p.want_beta)) continue;
    if constexpr (G > 32) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t c = (i * G + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < p.dim) part[c + j] = acc[i][j];
      }
    } else {
      // The row groups add into s_col one after another: a fixed order.
      if constexpr (VEC > 1) asm volatile("cp.async.wait_all;\n" ::: "memory");
      for (int t = 0; t < RPB; ++t) {
        __syncthreads();
        if (int(grp) == t) {
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const uint32_t c = (i * G + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s_col[c + j] = (t ? s_col[c + j] : 0.f) + acc[i][j];
          }
        }
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < p.dim; c += T) part[c] = s_col[c];
      __syncthreads();
    }
    part += p.dim;
  }
}

// Long rows: one block per row, grad_x only.
template <typename E, int VEC>
__global__ void __launch_bounds__(kNormLongThreads)
k_norm_bwd_long(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  __shared__ float s_sum[2][32];
  constexpr int G = kNormLongThreads;
  const uint32_t row = blockIdx.x;
  int64_t off[kMaxOperands];
  norm_row(p.rows, row, off);
  const E* g = static_cast<const E*>(p.in[0]) + off[0];
  const E* x = static_cast<const E*>(p.in[1]) + off[1];
  E* o = static_cast<E*>(p.out) + off[kSlotOut];
  const int64_t gs = VEC > 1 ? 1 : p.inner_stride[0];
  const int64_t xs = VEC > 1 ? 1 : p.inner_stride[1];
  const int64_t os = VEC > 1 ? 1 : p.inner_stride[kSlotOut];
  pdl_wait();
  const float mean = p.mean_in[row], rstd = p.rstd_in[row];
  float sq = 0.f, sqx = 0.f;
  for (uint64_t c = threadIdx.x * VEC; c < p.dim; c += G * VEC) {
    float gv[VEC], xv[VEC], ga[VEC];
    norm_load<E, VEC>(g + int64_t(c) * gs, gv);
    norm_load<E, VEC>(x + int64_t(c) * xs, xv);
    norm_affine<E, VEC>(p.gamma, p.gamma_stride, p.affine_vec, uint32_t(c), 1.f, ga);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float q = gv[j] * ga[j];
      sq += q;
      sqx = __fmaf_rn(q, (xv[j] - mean) * rstd, sqx);
    }
  }
  const float m1 = __fmul_rn(norm_sum<G>(sq, s_sum[0]), p.inv_dim);
  const float m2 = __fmul_rn(norm_sum<G>(sqx, s_sum[1]), p.inv_dim);
  for (uint64_t c = threadIdx.x * VEC; c < p.dim; c += G * VEC) {
    float gv[VEC], xv[VEC], ga[VEC];
    norm_load<E, VEC>(g + int64_t(c) * gs, gv);
    norm_load<E, VEC>(x + int64_t(c) * xs, xv);
    norm_affine<E, VEC>(p.gamma, p.gamma_stride, p.affine_vec, uint32_t(c), 1.f, ga);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      gv[j] = rstd * __fmaf_rn(-((xv[j] - mean) * rstd), m2, gv[j] * ga[j] - m1);
    norm_store<E, VEC>(o + int64_t(c) * os, gv);
  }
}

// Long rows: column sums.  A block takes 32 columns (lanes) and an equal run
// of the rows, one row per warp at a time; warps are added in order.
template <typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_sums(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  __shared__ float s_acc[2][kNormThreads / 32][32];
  const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint64_t c = uint64_t(blockIdx.x) * kNormSumCols + lane;
  const uint64_t lo = uint64_t(blockIdx.y) * p.nrow / gridDim.y;
  const uint64_t hi = uint64_t(blockIdx.y + 1) * p.nrow / gridDim.y;
  pdl_wait();
  float ag = 0.f, ab = 0.f;
  if (c < p.dim) {
    for (uint64_t r = lo + w; r < hi; r += kNormThreads / 32) {
      int64_t off[kMaxOperands];
      norm_row(p.rows, uint32_t(r), off);
      const float g = norm_ld(static_cast<const E*>(p.in[0]) + off[0] + int64_t(c) * p.inner_stride[0]);
      const float x = norm_ld(static_cast<const E*>(p.in[1]) + off[1] + int64_t(c) * p.inner_stride[1]);
      ag = __fmaf_rn(g, (x - p.mean_in[r]) * p.rstd_in[r], ag);
      ab += g;
    }
  }
  s_acc[0][w][lane] = ag;
  s_acc[1][w][lane] = ab;
  __syncthreads();
  if (w == 0 && c < p.dim) {
    ag = ab = 0.f;
#pragma unroll
    for (int k = 0; k < kNormThreads / 32; ++k) {
      ag += s_acc[0][k][lane];
      ab += s_acc[1][k][lane];
    }
    float* part = p.partial + uint64_t(blockIdx.y) * (p.want_gamma + p.want_beta) * p.dim;
    if (p.want_gamma) { part[c] = ag; part += p.dim; }
    if (p.want_beta) part[c] = ab;
  }
}

}  // namespace zr
