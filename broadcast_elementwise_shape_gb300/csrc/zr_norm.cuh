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
// backward read g and x and write grad_x.  So a row is read once (the variance
// is the two-pass one, from the differences, at no cost in traffic): G lanes
// hold a row of up to 32 columns each.  G = 8 for very short rows, a warp up to
// 1024 columns, then 2, 4 or 8 warps up to 8192.  Longer rows loop over the
// row, whose re-reads come from L1 and L2.
//
// The grid is persistent and what it needs is bytes in flight: rows are copied
// into a shared-memory ring p.stages - 1 rows ahead (cp.async, no registers).
// VEC > 1 (rows that start at 16-byte boundaries): each lane copies the vectors
// it will read itself, so no lane reads another's and there is no barrier.
// VEC = 1 with p.raw (rows of neighbouring elements at any address): the ring
// holds the aligned 16-byte granules around the row, and lanes read elements
// from there.  VEC = 1 without (strided rows): the elements are gathered into
// the ring by plain loads.  A lane's columns are the same for
// every row it meets, so gamma and beta stay in its registers, and in the
// backward the two column sums build up there; each block adds its row groups
// in a fixed order and writes one partial row, and the library's second pass
// adds the partials in order.  No atomics: the order is a function of the
// shape.  Arithmetic goes in pairs through the packed binary32 instructions,
// each lane of which rounds as the scalar one does.

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

// Barrier over the lanes of a row group.
template <int G>
__device__ __forceinline__ void norm_sync() {
  if constexpr (G <= 32) __syncwarp();
  else if constexpr (G == kNormThreads) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x) / G), "n"(G) : "memory");
}
// Sum over the G lanes of a row group.  G <= 32: butterflies, every lane gets
// the same bits.  More: warps by butterfly, then the warps' sums in order from
// s (one float per warp of the block, not reused before the next barrier).
template <int G>
__device__ __forceinline__ float norm_sum(float v, float* s) {
#pragma unroll
  for (int m = (G < 32 ? G : 32) / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    if constexpr (G > kNormThreads) __syncthreads();
    else norm_sync<G>();
    const float* t = s + threadIdx.x / G * (G / 32);
    v = t[0];
#pragma unroll
    for (int w = 1; w < G / 32; ++w) v += t[w];
  }
  return v;
}

// ------------------------------------------------------------------ the ring

__device__ __forceinline__ void norm_cp16(uint4* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void norm_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
// All copies but those of the last n commits (0, 1 or 2) have landed.
__device__ __forceinline__ void norm_wait(uint32_t n) {
  if (n == 2) asm volatile("cp.async.wait_group 2;\n" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
  else asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}
// Copies the granules around the `bytes` bytes at src into a slot whose start
// stands for src rounded down to 16 bytes.  Nothing before `base` or past the
// row is read: a first granule that begins before base goes element by element,
// the last one by its size.
template <typename E, int G>
__device__ __forceinline__ void norm_raw(uint4* slot, const E* src, const void* base, uint32_t bytes,
                                         uint32_t lane) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(src);
  const uintptr_t lo = at & ~uintptr_t(15), hi = at + bytes;
  for (uint32_t k = lane; lo + 16 * k < hi; k += G) {
    const uintptr_t g = lo + 16 * k;
    if (g < reinterpret_cast<uintptr_t>(base)) {
      E* dst = reinterpret_cast<E*>(reinterpret_cast<char*>(slot) + (at - lo));
      for (uint32_t e = 0; at + e * sizeof(E) < (g + 16 < hi ? g + 16 : hi); ++e) dst[e] = src[e];
    } else if (g + 16 <= hi) {
      norm_cp16(slot + k, reinterpret_cast<const void*>(g));
    } else {
      const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(slot + k));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(g), "r"(uint32_t(hi - g))
                   : "memory");
    }
  }
}
// Column h of a lane's i-th pair (VEC = 1): neighbours for 2-byte elements,
// G apart for 4-byte ones, so that a warp's shared-memory reads and its stores
// are contiguous.
template <typename E, int G>
__device__ __forceinline__ uint32_t norm_col(int i, int h, uint32_t lane) {
  return sizeof(E) == 2 ? 2 * (i * G + lane) + h : (2 * i + h) * G + lane;
}
// Puts a row into its slot (VEC = 1).
template <typename E, int G>
__device__ __forceinline__ void norm_gather(const NormPlan& p, uint4* slot, int in, int64_t off,
                                            uint32_t lane) {
  const E* src = static_cast<const E*>(p.in[in]) + off;
  if (p.raw) {
    norm_raw<E, G>(slot, src, p.in[in], p.dim * uint32_t(sizeof(E)), lane);
  } else {
    E* dst = reinterpret_cast<E*>(slot);
#pragma unroll 4
    for (uint32_t c = lane; c < p.dim; c += G) dst[c] = src[int64_t(c) * p.inner_stride[in]];
  }
}
// Where the row's first element is in its slot.
template <typename E>
__device__ __forceinline__ const E* norm_start(const NormPlan& p, const uint4* slot, int in, int64_t off) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const E*>(p.in[in]) + off);
  return reinterpret_cast<const E*>(slot) + (p.raw ? (at & 15) / sizeof(E) : 0);
}
// The lane's i-th pair of a row in its slot, `pad` past its end.
template <typename E, int G>
__device__ __forceinline__ F2 norm_pair(const NormPlan& p, const E* row, int i, uint32_t lane, float pad) {
  float f[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = norm_col<E, G>(i, h, lane);
    f[h] = c < p.dim ? norm_ld(row + c) : pad;
  }
  return f2_pack(f[0], f[1]);
}
template <typename E, int G>
__device__ __forceinline__ void norm_put_pair(const NormPlan& p, E* row, int64_t stride, int i,
                                              uint32_t lane, F2 v) {
  float f[2];
  f2_unpack(v, f[0], f[1]);
  const uint32_t c = norm_col<E, G>(i, 0, lane);
  if constexpr (sizeof(E) == 2) {
    if (p.out_pairs && c + 1 < p.dim) {  // rows of y start at 4-byte boundaries
      *reinterpret_cast<__nv_bfloat162*>(row + c) = __floats2bfloat162_rn(f[0], f[1]);
      return;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t ch = norm_col<E, G>(i, h, lane);
    if (ch < p.dim) st1(row + int64_t(ch) * stride, f[h]);
  }
}
// gamma or beta of the lane's i-th item (VEC elements, or a pair).
template <typename E, int VEC, int G>
__device__ __forceinline__ void norm_affine_item(const NormPlan& p, const void* base, int64_t stride,
                                                 int i, uint32_t lane, float none, F2* v) {
  constexpr int N = VEC > 1 ? VEC : 2;
  float f[N];
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] = 0.f;
  if constexpr (VEC > 1) {
    const uint32_t c = (i * G + lane) * VEC;
    if (c < p.dim) norm_affine<E, VEC>(base, stride, p.affine_vec, c, none, f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = norm_col<E, G>(i, h, lane);
      if (c < p.dim) norm_affine<E, 1>(base, stride, 0, c, none, &f[h]);
    }
  }
#pragma unroll
  for (int j = 0; j < N / 2; ++j) v[j] = f2_pack(f[2 * j], f[2 * j + 1]);
}
// The VEC elements of a 16-byte slot as pairs.
template <typename E>
__device__ __forceinline__ void norm_pairs(const uint4* slot, F2* v) {
  if constexpr (sizeof(E) == 4) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(slot);
    v[0].v = q.x;
    v[1].v = q.y;
  } else {
    const uint4 q = *slot;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
}
template <typename E, int VEC>
__device__ __forceinline__ void norm_store_pairs(E* p, const F2* v) {
  float f[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) f2_unpack(v[i], f[2 * i], f[2 * i + 1]);
  norm_store<E, VEC>(p, f);
}
__device__ __forceinline__ float f2_sum(F2 a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}

template <typename E, int VEC, int G, int NI>
__global__ void __launch_bounds__(kNormThreads, norm_occ(NI * VEC))
k_norm_fwd(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  constexpr int RPB = kNormThreads / G;           // rows per block per step
  constexpr int H = VEC > 1 ? VEC / 2 : 1;        // pairs per item
  constexpr int NP = VEC > 1 ? NI : NI / 2;       // items per lane: vectors, or pairs
  __shared__ float s_sum[2][2][32];
  extern __shared__ uint4 s_ring[];  // [stage][row group][p.slot]
  const uint32_t lane = threadIdx.x % G, grp = threadIdx.x / G;
  const uint64_t step = uint64_t(gridDim.x) * RPB;
  const uint64_t first = uint64_t(blockIdx.x) * RPB + grp;
  const uint32_t S = p.stages;
  auto slot = [&](uint32_t stage) { return s_ring + (uint64_t(stage) * RPB + grp) * p.slot; };
  auto fetch = [&](uint32_t stage, uint64_t row) {
    if (row < p.nrow) {
      int64_t off[kMaxOperands];
      norm_row(p.rows, uint32_t(row), off);
      if constexpr (VEC > 1) {
        const E* x = static_cast<const E*>(p.in[0]) + off[0];
        uint4* q = slot(stage) + lane;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if ((i * G + lane) * VEC < p.dim) norm_cp16(q + i * G, x + (i * G + lane) * VEC);
      } else {
        norm_gather<E, G>(p, slot(stage), 0, off[0], lane);
      }
    }
    norm_commit();
  };
  pdl_wait();
  for (uint32_t k = 0; k + 1 < S; ++k) fetch(k, first + k * step);
  F2 ga[NP][H], be[NP][H];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    norm_affine_item<E, VEC, G>(p, p.gamma, p.gamma_stride, i, lane, 1.f, ga[i]);
    norm_affine_item<E, VEC, G>(p, p.beta, p.beta_stride, i, lane, 0.f, be[i]);
  }
  uint32_t stage = 0, ahead = S - 1, flip = 0;
  for (uint64_t r0 = uint64_t(blockIdx.x) * RPB; r0 < p.nrow; r0 += step) {
    const uint64_t row = r0 + grp;
    const bool live = row < p.nrow;
    int64_t off[kMaxOperands];
    norm_row(p.rows, live ? uint32_t(row) : 0, off);
    if constexpr (VEC > 1) {
      fetch(ahead, row + (S - 1) * step);
      norm_wait(S - 1);
    } else {
      // Lanes read each other's copies: the slot filled next is the last row's,
      // which every lane has read once all of them are here.
      norm_wait(S - 2);
      norm_sync<G>();
      fetch(ahead, row + (S - 1) * step);
    }
    const E* src = norm_start<E>(p, slot(stage), 0, off[0]);  // VEC = 1
    F2 v[NP][H];
    F2 acc = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (VEC > 1) {
        if (live && (i * G + lane) * VEC < p.dim) {
          norm_pairs<E>(slot(stage) + lane + i * G, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < H; ++j) v[i][j] = f2_splat(0.f);
        }
      } else {
        v[i][0] = live ? norm_pair<E, G>(p, src, i, lane, 0.f) : f2_splat(0.f);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) acc = f2_add(acc, v[i][j]);
    }
    const float mean = __fmul_rn(norm_sum<G>(f2_sum(acc), s_sum[flip][0]), p.inv_dim);
    const F2 minus = f2_splat(-mean);
    acc = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (VEC > 1) {
        if ((i * G + lane) * VEC < p.dim) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            v[i][j] = f2_add(v[i][j], minus);
            acc = f2_fma(v[i][j], v[i][j], acc);
          }
        }
      } else {
        float f[2];
        f2_unpack(f2_add(v[i][0], minus), f[0], f[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (norm_col<E, G>(i, h, lane) >= p.dim) f[h] = 0.f;  // past the row's end
        v[i][0] = f2_pack(f[0], f[1]);
        acc = f2_fma(v[i][0], v[i][0], acc);
      }
    }
    const float var = __fmul_rn(norm_sum<G>(f2_sum(acc), s_sum[flip][1]), p.inv_dim);
    flip ^= 1;  // the next row writes the other pair: one barrier lies between
    const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
    if (live) {
      if (lane == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
      }
      E* y = static_cast<E*>(p.out) + off[kSlotOut];
      const F2 r2 = f2_splat(rstd);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
#pragma unroll
        for (int j = 0; j < H; ++j) v[i][j] = f2_fma(f2_mul(v[i][j], r2), ga[i][j], be[i][j]);
        if constexpr (VEC > 1) {
          if ((i * G + lane) * VEC < p.dim) norm_store_pairs<E, VEC>(y + (i * G + lane) * VEC, v[i]);
        } else {
          norm_put_pair<E, G>(p, y, p.inner_stride[kSlotOut], i, lane, v[i][0]);
        }
      }
    }
    if (++stage == S) stage = 0;
    if (++ahead == S) ahead = 0;
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

// A row waits in the ring and is read twice from there, once for its two means
// and the column sums, once for grad_x: kept in registers instead it took 222
// of them, 8 warps per SM, and [65536, 1024] bf16 137 us; 60 now.
template <typename E, int VEC, int G, int NI>
__global__ void __launch_bounds__(kNormThreads, norm_occ(NI * VEC))
k_norm_bwd(const __grid_constant__ NormPlan p) {
  pdl_trigger();
  constexpr int T = kNormThreads;
  constexpr int RPB = T / G;           // rows per block per step
  constexpr int W = G * NI * VEC;      // columns the lanes cover
  constexpr int H = VEC > 1 ? VEC / 2 : 1;
  constexpr int NP = VEC > 1 ? NI : NI / 2;
  extern __shared__ uint4 s_ring[];    // [stage][row group][g, x][p.slot]; then column sums
  __shared__ float s_sum[2][2][32];
  const uint32_t lane = threadIdx.x % G, grp = threadIdx.x / G;
  F2 acc_g[NP][H], acc_b[NP][H], gam[NP][H];
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < H; ++j) acc_g[i][j] = acc_b[i][j] = f2_splat(0.f);
  const uint64_t step = uint64_t(gridDim.x) * RPB;
  const uint64_t first = uint64_t(blockIdx.x) * RPB + grp;
  const uint32_t S = p.stages;
  auto slot = [&](uint32_t stage, int a) {
    return s_ring + ((uint64_t(stage) * RPB + grp) * 2 + a) * p.slot;
  };
  auto fetch = [&](uint32_t stage, uint64_t row) {
    if (row < p.nrow) {
      int64_t off[kMaxOperands];
      norm_row(p.rows, uint32_t(row), off);
      if constexpr (VEC > 1) {
        const E* g = static_cast<const E*>(p.in[0]) + off[0];
        const E* x = static_cast<const E*>(p.in[1]) + off[1];
        uint4* sg = slot(stage, 0) + lane;
        uint4* sx = slot(stage, 1) + lane;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t c = (i * G + lane) * VEC;
          if (c < p.dim) {
            norm_cp16(sg + i * G, g + c);
            norm_cp16(sx + i * G, x + c);
          }
        }
      } else {
        norm_gather<E, G>(p, slot(stage, 0), 0, off[0], lane);
        norm_gather<E, G>(p, slot(stage, 1), 1, off[1], lane);
      }
    }
    norm_commit();
  };
  pdl_wait();
  for (uint32_t k = 0; k + 1 < S; ++k) fetch(k, first + k * step);
  float mean = first < p.nrow ? p.mean_in[first] : 0.f;
  float rstd = first < p.nrow ? p.rstd_in[first] : 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    norm_affine_item<E, VEC, G>(p, p.gamma, p.gamma_stride, i, lane, 1.f, gam[i]);
  uint32_t flip = 0, stage = 0, ahead = S - 1;
  for (uint64_t r0 = uint64_t(blockIdx.x) * RPB; r0 < p.nrow; r0 += step) {
    const uint64_t row = r0 + grp;
    const bool live = row < p.nrow;
    // The next row's statistics, and the row S - 1 steps on.
    const float mean_next = row + step < p.nrow ? p.mean_in[row + step] : 0.f;
    const float rstd_next = row + step < p.nrow ? p.rstd_in[row + step] : 0.f;
    int64_t off[kMaxOperands];
    norm_row(p.rows, live ? uint32_t(row) : 0, off);
    if constexpr (VEC > 1) {
      fetch(ahead, row + (S - 1) * step);
      norm_wait(S - 1);
    } else {
      // Lanes read each other's copies: the slot filled next is the last row's,
      // which every lane has read once all of them are here.
      norm_wait(S - 2);
      norm_sync<G>();
      fetch(ahead, row + (S - 1) * step);
    }
    const F2 minus = f2_splat(-mean), r2 = f2_splat(rstd);
    const E* rg = norm_start<E>(p, slot(stage, 0), 0, off[0]);  // VEC = 1
    const E* rx = norm_start<E>(p, slot(stage, 1), 1, off[1]);
    auto load = [&](int i, F2* gv, F2* xv) {
      if constexpr (VEC > 1) {
        norm_pairs<E>(slot(stage, 0) + lane + i * G, gv);
        norm_pairs<E>(slot(stage, 1) + lane + i * G, xv);
      } else {  // past the row's end: a gradient of 0 at the mean, which adds nothing
        gv[0] = norm_pair<E, G>(p, rg, i, lane, 0.f);
        xv[0] = norm_pair<E, G>(p, rx, i, lane, mean);
      }
    };
    F2 sq = f2_splat(0.f), sqx = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (live && (VEC == 1 || (i * G + lane) * VEC < p.dim)) {
        F2 gv[H], xv[H];
        load(i, gv, xv);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const F2 xh = f2_mul(f2_add(xv[j], minus), r2);
          acc_b[i][j] = f2_add(acc_b[i][j], gv[j]);
          acc_g[i][j] = f2_fma(gv[j], xh, acc_g[i][j]);
          const F2 q = f2_mul(gv[j], gam[i][j]);
          sq = f2_add(sq, q);
          sqx = f2_fma(q, xh, sqx);
        }
      }
    }
    if (p.out) {
      const float m1 = __fmul_rn(norm_sum<G>(f2_sum(sq), s_sum[flip][0]), p.inv_dim);
      const float m2 = __fmul_rn(norm_sum<G>(f2_sum(sqx), s_sum[flip][1]), p.inv_dim);
      flip ^= 1;  // the next row writes the other pair: one barrier lies between
      // grad_x = g (gamma rstd) - (xh (m2 rstd) + m1 rstd)
      const F2 a = f2_splat(-__fmul_rn(m2, rstd)), b = f2_splat(-__fmul_rn(m1, rstd));
      E* o = static_cast<E*>(p.out) + off[kSlotOut];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (live && (VEC == 1 || (i * G + lane) * VEC < p.dim)) {
          F2 gv[H], xv[H];
          load(i, gv, xv);
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const F2 xh = f2_mul(f2_add(xv[j], minus), r2);
            xv[j] = f2_fma(gv[j], f2_mul(gam[i][j], r2), f2_fma(xh, a, b));
          }
          if constexpr (VEC > 1) norm_store_pairs<E, VEC>(o + (i * G + lane) * VEC, xv);
          else norm_put_pair<E, G>(p, o, p.inner_stride[kSlotOut], i, lane, xv[0]);
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
  // Every row group's sums side by side (the ring's copies are all in and
  // read), then each column's in the groups' order.
  float* s_col = reinterpret_cast<float*>(s_ring);  // [row group][W]
  if constexpr (RPB > 1) {
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    F2(&acc)[NP][H] = k == 0 ? acc_g : acc_b;
    if (!(k == 0 ? p.want_gamma : p.want_beta)) continue;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
#pragma unroll
      for (int j = 0; j < H; ++j) {
        float v[2];
        f2_unpack(acc[i][j], v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t c = VEC > 1 ? (i * G + lane) * VEC + 2 * j + h : norm_col<E, G>(i, h, lane);
          if constexpr (RPB > 1) s_col[grp * W + c] = v[h];
          else if (c < p.dim) part[c] = v[h];
        }
      }
    }
    if constexpr (RPB > 1) {
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < p.dim; c += T) {
        float t = s_col[c];
#pragma unroll
        for (int r = 1; r < RPB; ++r) t += s_col[r * W + c];
        part[c] = t;
      }
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
