// zr_attn_any.cu — causal attention in binary32 arithmetic: the tensors that the
// tensor-core kernels do not take (zr_attn.cu): binary32 heads of over 64 elements,
// bfloat16 ones of over 128, at odd addresses or of odd sizes, negative scales.
//
// One pass over the keys with a row's running maximum and sum: a tile of 64
// queries stays, tiles of keys and values go past, and no score is ever
// stored.  The backward computes the scores again, twice: a tile of keys with
// all queries that see it for grad_k and grad_v, a tile of queries with all its
// keys for grad_q.  That is seven products for the five it cannot do without,
// and in return every gradient is summed in one place, in a fixed order.
//
// Bound by the binary32 multiply-adds and the reads from shared memory that feed
// them ([1, 2048] tokens of 16 heads of 128, 467 us forward: 37 TFLOP/s of 74).  256 threads hold a 64 x 64 tile of
// scores as 4 x 4 each, rows and columns 16 apart, so that the 16-byte reads of
// the operands along the elements meet no bank twice (rows are padded by 16
// bytes); 16 reads feed 64 multiply-adds, in pairs (two per instruction).  What
// is exchanged, the weights, goes from the threads of one half warp to the same
// threads: a row of the tile belongs to 16 lanes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zr_attn.h"
#include "zr_kernels.cuh"
#include "zr_launch.h"
#include "zr_tc.cuh"

namespace zr {
namespace {

constexpr uint32_t kAnyRows = 64;   // rows of the tile that stays

__device__ __forceinline__ float any_load(const float* p) { return *p; }
__device__ __forceinline__ float any_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void any_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void any_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ void rows_load(const float* p, float (&x)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
}
__device__ __forceinline__ void rows_load(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
}

// ROWS rows from `row0` of a head into shared memory, DP elements each, zero
// behind the sequence's end and the head's.
template <typename E, int DP, int ROWS>
__device__ __forceinline__ void any_fetch(float* to, const AttnPlan& p, const AttnView& x, uint32_t batch, uint32_t head,
                                          uint32_t start, uint32_t row0, uint32_t len) {
  const E* base = static_cast<const E*>(x.p) + int64_t(batch) * x.batch + int64_t(head) * x.head + int64_t(start) * x.token;
  constexpr int V = 16 / int(sizeof(E));
  if (p.vec) {
    constexpr int kPer = DP / V;
    for (int i = threadIdx.x; i < ROWS * kPer; i += kThreads) {
      const uint32_t r = uint32_t(i) / kPer, c = (uint32_t(i) - r * kPer) * V;
      float* o = to + r * (DP + 4) + c;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (row0 + r < len && c < p.dim) w = *reinterpret_cast<const uint4*>(base + int64_t(row0 + r) * x.token + c);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      if constexpr (V == 4) {
        *reinterpret_cast<uint4*>(o) = w;
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint4*>(o + 4 * h) = make_uint4(u[2 * h] << 16, u[2 * h] & 0xFFFF0000u, u[2 * h + 1] << 16,
                                                            u[2 * h + 1] & 0xFFFF0000u);
      }
    }
  } else {
    for (int i = threadIdx.x; i < ROWS * DP; i += kThreads) {
      const uint32_t r = uint32_t(i) / DP, c = uint32_t(i) - r * DP;
      float f = 0.f;
      if (row0 + r < len && c < p.dim) f = any_load(base + int64_t(row0 + r) * x.token + int64_t(c) * x.elem);
      to[r * (DP + 4) + c] = f;
    }
  }
}

// acc[i][j] = sum over the elements of A[ty + 16 i] B[tx + 16 j].
template <int DP, int M, int N>
__device__ __forceinline__ void any_scores(const float* a, const float* b, float (&acc)[M][N]) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  F2 sum[M][N];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) sum[i][j] = f2_splat(0.f);
  a += ty * (DP + 4);
  b += tx * (DP + 4);
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 x[M], y[N];
#pragma unroll
    for (int i = 0; i < M; ++i) x[i] = *reinterpret_cast<const float4*>(a + i * 16 * (DP + 4) + d);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = *reinterpret_cast<const float4*>(b + j * 16 * (DP + 4) + d);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        sum[i][j] = f2_fma(f2_pack(x[i].x, x[i].y), f2_pack(y[j].x, y[j].y), sum[i][j]);
        sum[i][j] = f2_fma(f2_pack(x[i].z, x[i].w), f2_pack(y[j].z, y[j].w), sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float lo, hi;
      f2_unpack(sum[i][j], lo, hi);
      acc[i][j] = lo + hi;
    }
}

// acc[i] (elements 4 tx + 64 c) += sum over K of w[ty + 16 i][k] B[k].
template <int DP, int M, int K>
__device__ __forceinline__ void any_sum(const float* w, const float* b, F2 (&acc)[M][DP / 64][2]) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  constexpr int kPitch = K + 4;       // of the weights' tile
  w += ty * kPitch;
  b += tx * 4;
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 x[M];
#pragma unroll
    for (int i = 0; i < M; ++i) x[i] = *reinterpret_cast<const float4*>(w + i * 16 * kPitch + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const float4 y = *reinterpret_cast<const float4*>(b + (k + e) * (DP + 4) + c * 64);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const F2 f = f2_splat(e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w);
          acc[i][c][0] = f2_fma(f, f2_pack(y.x, y.y), acc[i][c][0]);
          acc[i][c][1] = f2_fma(f, f2_pack(y.z, y.w), acc[i][c][1]);
        }
      }
    }
  }
}

// Rows ty + 16 i of a result, times `by[i]`; low: the rounding error besides.
template <typename E, int DP, int M>
__device__ __forceinline__ void any_write(const AttnPlan& p, const AttnView& x, void* low, uint32_t batch, uint32_t head,
                                          uint32_t heads, uint32_t start, uint32_t row0, uint32_t len,
                                          const F2 (&acc)[M][DP / 64][2], const float* by) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const uint32_t r = row0 + ty + 16 * i;
    if (r >= len) continue;
    const int64_t token = int64_t(start) + r;
    E* o = static_cast<E*>(const_cast<void*>(x.p)) + int64_t(batch) * x.batch + int64_t(head) * x.head + token * x.token;
    E* l = static_cast<E*>(low) + ((int64_t(batch) * p.tokens + token) * heads + head) * p.dim;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const uint32_t d = 4 * tx + 64 * c;
      float f[4];
      f2_unpack(acc[i][c][0], f[0], f[1]);
      f2_unpack(acc[i][c][1], f[2], f[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (d + e >= p.dim) continue;
        const float y = f[e] * by[i];
        any_store(o + int64_t(d + e) * x.elem, y);
        if (sizeof(E) == 2 && low) any_store(l + d + e, y - __bfloat162float(__float2bfloat16_rn(y)));
      }
    }
  }
}

// Reductions over the 16 lanes that share a row.
__device__ __forceinline__ float any_max16(float x) {
#pragma unroll
  for (int d = 8; d; d /= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  return x;
}
__device__ __forceinline__ float any_add16(float x) {
#pragma unroll
  for (int d = 8; d; d /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

// Heads of 65 to 128 elements bring keys and values through one room in shared
// memory, one after the other: two CTAs fit an SM, and one computes while the other
// loads ([1, 2048] tokens of 16 heads of 128, 488 us with a room each).
template <int DP>
constexpr bool kOneRoom = DP == 128;
// blockIdx.x = slot * heads + head.
template <typename E, int DP>
__global__ void __launch_bounds__(kThreads, DP == 128 ? 2 : 1) k_attn_any_fwd(const __grid_constant__ AttnPlan p) {
  extern __shared__ float s_f[];
  float* sq = s_f;
  float* sk = sq + kAnyRows * (DP + 4);
  float* sv = kOneRoom<DP> ? sk : sk + 64 * (DP + 4);
  float* sw = sv + 64 * (DP + 4);
  pdl_trigger();
  pdl_wait();
  const uint32_t slot = blockIdx.x / p.heads, head = blockIdx.x - slot * p.heads, kvh = head / p.group;
  const AttnTile t = attn_tile(p, slot, false);
  if (!t.live) return;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const uint32_t row0 = t.tile * kAnyRows;
  any_fetch<E, DP, 64>(sq, p, p.q, t.batch, head, t.start, row0, t.len);
  F2 acc[4][DP / 64][2];
  float top[4], sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) acc[i][c][0] = acc[i][c][1] = f2_splat(0.f);
  }
  for (uint32_t k0 = 0; k0 <= row0; k0 += 64) {
    __syncthreads();
    any_fetch<E, DP, 64>(sk, p, p.k, t.batch, kvh, t.start, k0, t.len);
    if (!kOneRoom<DP>) any_fetch<E, DP, 64>(sv, p, p.v, t.batch, kvh, t.start, k0, t.len);
    __syncthreads();
    float s[4][4];
    any_scores<DP>(sq, sk, s);
    if (kOneRoom<DP>) {
      __syncthreads();
      any_fetch<E, DP, 64>(sv, p, p.v, t.batch, kvh, t.start, k0, t.len);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = row0 + ty + 16 * i;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = k0 + tx + 16 * j;
        s[i][j] = c <= r ? s[i][j] * p.scale : -INFINITY;
        m = fmaxf(m, s[i][j]);
      }
      m = fmaxf(top[i], any_max16(m));
      const float base = m == -INFINITY ? 0.f : m;
      const float keep = ex2_full((top[i] - base) * kLog2e);
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = ex2_full((s[i][j] - base) * kLog2e);
        add += w;
        sw[(ty + 16 * i) * 68 + tx + 16 * j] = w;
      }
      sum[i] = __fmaf_rn(sum[i], keep, any_add16(add));
      top[i] = m;
      const F2 f = f2_splat(keep);
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        acc[i][c][0] = f2_mul(acc[i][c][0], f);
        acc[i][c][1] = f2_mul(acc[i][c][1], f);
      }
    }
    if (kOneRoom<DP>) __syncthreads();
    else __syncwarp();
    any_sum<DP, 4, 64>(sw, sv, acc);
  }
  float by[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    by[i] = 1.f / sum[i];
    const uint32_t r = row0 + ty + 16 * i;
    if (p.lse && tx == 0 && r < t.len)
      p.lse[(int64_t(t.batch) * p.tokens + t.start + r) * p.heads + head] = top[i] + logf(sum[i]);
  }
  any_write<E, DP>(p, p.o, p.low, t.batch, head, p.heads, t.start, row0, t.len, acc, by);
}

// delta = sum of grad_out * out, and lse2, of rows (batch, token, head).  Eight
// lanes take kRowsEach rows one behind the other, 16 bytes a lane where the
// tensors allow it, all under way before the first is used.
constexpr int kRowsEach = 4;
template <typename E>
__global__ void __launch_bounds__(kThreads) k_attn_rows(const __grid_constant__ AttnPlan p) {
  constexpr uint32_t V = 16 / sizeof(E);
  pdl_wait();
  pdl_trigger();  // behind the wait: k_attn_split may start beside this kernel, its operands are there
  const uint32_t lane = threadIdx.x % 8;
  const uint32_t n = p.batch * p.tokens * p.heads;
  const uint32_t first = (blockIdx.x * (kThreads / 8) + threadIdx.x / 8) * kRowsEach;
  if (first - threadIdx.x / 8 * kRowsEach >= n) return;
  const bool low = sizeof(E) == 2 && p.low;
  const E *o[kRowsEach], *g[kRowsEach];
  float sum[kRowsEach];
  int64_t at[kRowsEach];
  uint32_t i = first < n ? first : n - 1, t = i / p.heads, head = i - t * p.heads, b = t / p.tokens;
  t -= b * p.tokens;
  uint32_t row[kRowsEach];
#pragma unroll
  for (int u = 0; u < kRowsEach; ++u) {
    row[u] = i;
    o[u] = static_cast<const E*>(p.o.p) + int64_t(b) * p.o.batch + int64_t(t) * p.o.token + int64_t(head) * p.o.head;
    g[u] = static_cast<const E*>(p.go.p) + int64_t(b) * p.go.batch + int64_t(t) * p.go.token + int64_t(head) * p.go.head;
    at[u] = (int64_t(b) * p.heads + head) * p.row_pitch + t;
    sum[u] = 0.f;
    if (i + 1 < n) {  // the next row; the last one again behind the end
      ++i;
      if (++head == p.heads) {
        head = 0;
        if (++t == p.tokens) {
          t = 0;
          ++b;
        }
      }
    }
  }
  const auto low_of = [&](int u) { return static_cast<const E*>(p.low) + int64_t(row[u]) * p.dim; };
  if (p.o_wide) {
    for (uint32_t d = lane * V; d < p.dim; d += 8 * V) {
      float x[kRowsEach][V], y[kRowsEach][V], z[kRowsEach][V];
#pragma unroll
      for (int u = 0; u < kRowsEach; ++u) {
        rows_load(o[u] + d, x[u]);
        rows_load(g[u] + d, y[u]);
        if (low) rows_load(low_of(u) + d, z[u]);
      }
#pragma unroll
      for (int u = 0; u < kRowsEach; ++u)
#pragma unroll
        for (uint32_t k = 0; k < V; ++k) sum[u] = __fmaf_rn(low ? x[u][k] + z[u][k] : x[u][k], y[u][k], sum[u]);
    }
  } else {
    for (uint32_t d = lane; d < p.dim; d += 8) {
#pragma unroll
      for (int u = 0; u < kRowsEach; ++u) {
        float x = any_load(o[u] + int64_t(d) * p.o.elem);
        if (low) x += any_load(low_of(u) + d);
        sum[u] = __fmaf_rn(x, any_load(g[u] + int64_t(d) * p.go.elem), sum[u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsEach; ++u) {
#pragma unroll
    for (int d = 4; d; d /= 2) sum[u] += __shfl_xor_sync(0xFFFFFFFFu, sum[u], d);
    if (lane == uint32_t(u) && first + u < n && first + u >= first) {
      p.delta[at[u]] = sum[u];
      p.lse2[at[u]] = p.lse[row[u]] * kLog2e;
    }
  }
}

// Weight of a score, and of its gradient; lse2 is lse * log2(e).
__device__ __forceinline__ float any_weight(float s, float scale, float lse, bool sees) {
  return sees ? ex2_full((s * scale - lse) * kLog2e) : 0.f;
}

// grad_k and grad_v of a tile of 64 keys: all queries of the group's heads that
// see it, R at a time.  blockIdx.x = slot * kv_heads + kv head.
template <typename E, int DP, int R>
__global__ void __launch_bounds__(kThreads) k_attn_any_kv(const __grid_constant__ AttnPlan p) {
  extern __shared__ float s_f[];
  float* sk = s_f;
  float* sv = sk + 64 * (DP + 4);
  float* sq = sv + 64 * (DP + 4);
  float* sg = sq + R * (DP + 4);
  float* sw = sg + R * (DP + 4);      // [key][query]
  float* sd = sw + 64 * (R + 4);
  float* s_row = sd + 64 * (R + 4);  // lse and delta of R queries
  pdl_trigger();
  pdl_wait();
  const uint32_t slot = blockIdx.x / p.kv_heads, kvh = blockIdx.x - slot * p.kv_heads;
  const AttnTile t = attn_tile(p, slot, true);
  if (!t.live) return;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const uint32_t key0 = t.tile * 64;
  any_fetch<E, DP, 64>(sk, p, p.k, t.batch, kvh, t.start, key0, t.len);
  any_fetch<E, DP, 64>(sv, p, p.v, t.batch, kvh, t.start, key0, t.len);
  F2 gk[4][DP / 64][2], gv[4][DP / 64][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) gk[i][c][0] = gk[i][c][1] = gv[i][c][0] = gv[i][c][1] = f2_splat(0.f);
  for (uint32_t head = kvh * p.group; head < (kvh + 1) * p.group; ++head) {
    for (uint32_t q0 = key0; q0 < t.len; q0 += R) {
      __syncthreads();
      any_fetch<E, DP, R>(sq, p, p.q, t.batch, head, t.start, q0, t.len);
      any_fetch<E, DP, R>(sg, p, p.go, t.batch, head, t.start, q0, t.len);
      if (threadIdx.x < R && q0 + threadIdx.x < t.len) {
        const uint32_t row = t.start + q0 + threadIdx.x;
        s_row[threadIdx.x] = p.lse[(int64_t(t.batch) * p.tokens + row) * p.heads + head];
        s_row[R + threadIdx.x] = p.delta[(int64_t(t.batch) * p.heads + head) * p.row_pitch + row];
      }
      __syncthreads();
      float s[4][R / 16], d[4][R / 16];
      any_scores<DP>(sk, sq, s);
      any_scores<DP>(sv, sg, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < R / 16; ++j) {
          const uint32_t key = key0 + ty + 16 * i, c = tx + 16 * j, query = q0 + c;
          const bool sees = key <= query && query < t.len;
          const float w = any_weight(s[i][j], p.scale, s_row[c], sees);
          sw[(ty + 16 * i) * (R + 4) + c] = w;
          sd[(ty + 16 * i) * (R + 4) + c] = sees ? w * (d[i][j] - s_row[R + c]) : 0.f;
        }
      }
      __syncwarp();
      any_sum<DP, 4, R>(sw, sg, gv);
      any_sum<DP, 4, R>(sd, sq, gk);
    }
  }
  float one[4] = {1.f, 1.f, 1.f, 1.f}, by[4] = {p.scale, p.scale, p.scale, p.scale};
  if (p.want & 4) any_write<E, DP>(p, p.gv, nullptr, t.batch, kvh, p.kv_heads, t.start, key0, t.len, gv, one);
  if (p.want & 2) any_write<E, DP>(p, p.gk, nullptr, t.batch, kvh, p.kv_heads, t.start, key0, t.len, gk, by);
}

// grad_q of a tile of 64 queries: all keys it sees, R at a time.
// blockIdx.x = slot * heads + head.
template <typename E, int DP, int R>
__global__ void __launch_bounds__(kThreads) k_attn_any_q(const __grid_constant__ AttnPlan p) {
  extern __shared__ float s_f[];
  float* sq = s_f;
  float* sg = sq + 64 * (DP + 4);
  float* sk = sg + 64 * (DP + 4);
  float* sv = sk + R * (DP + 4);
  float* sd = sv + R * (DP + 4);
  pdl_trigger();
  pdl_wait();
  const uint32_t slot = blockIdx.x / p.heads, head = blockIdx.x - slot * p.heads, kvh = head / p.group;
  const AttnTile t = attn_tile(p, slot, false);
  if (!t.live) return;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const uint32_t row0 = t.tile * 64;
  any_fetch<E, DP, 64>(sq, p, p.q, t.batch, head, t.start, row0, t.len);
  any_fetch<E, DP, 64>(sg, p, p.go, t.batch, head, t.start, row0, t.len);
  F2 gq[4][DP / 64][2];
  float lse[4], delta[4], by[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = row0 + ty + 16 * i, row = t.start + r;
    lse[i] = delta[i] = 0.f;
    by[i] = p.scale;
    if (r < t.len) {
      lse[i] = p.lse[(int64_t(t.batch) * p.tokens + row) * p.heads + head];
      delta[i] = p.delta[(int64_t(t.batch) * p.heads + head) * p.row_pitch + row];
    }
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) gq[i][c][0] = gq[i][c][1] = f2_splat(0.f);
  }
  for (uint32_t k0 = 0; k0 < row0 + 64 && k0 < t.len; k0 += R) {
    __syncthreads();
    any_fetch<E, DP, R>(sk, p, p.k, t.batch, kvh, t.start, k0, t.len);
    any_fetch<E, DP, R>(sv, p, p.v, t.batch, kvh, t.start, k0, t.len);
    __syncthreads();
    float s[4][R / 16], d[4][R / 16];
    any_scores<DP>(sq, sk, s);
    any_scores<DP>(sg, sv, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < R / 16; ++j) {
        const uint32_t r = row0 + ty + 16 * i, c = tx + 16 * j;
        const bool sees = k0 + c <= r && r < t.len;
        const float w = any_weight(s[i][j], p.scale, lse[i], sees);
        sd[(ty + 16 * i) * (R + 4) + c] = sees ? w * (d[i][j] - delta[i]) : 0.f;
      }
    }
    __syncwarp();
    any_sum<DP, 4, R>(sd, sk, gq);
  }
  any_write<E, DP>(p, p.gq, nullptr, t.batch, head, p.heads, t.start, row0, t.len, gq, by);
}

template <typename E, int DP>
cudaError_t any_fwd(const AttnPlan& p, cudaStream_t s) {
  constexpr size_t smem = ((kOneRoom<DP> ? 2 : 3) * 64 * (DP + 4) + 64 * 68) * sizeof(float);
  const auto k = with_smem(k_attn_any_fwd<E, DP>, smem);
  return k ? launch_k(k, p.slots * p.heads, kThreads, smem, s, p) : cudaErrorInvalidValue;
}

template <typename E, int DP>
cudaError_t any_bwd(const AttnPlan& p, cudaStream_t s) {
  // Of heads over 128 elements half as many rows go past at a time, for room.
  constexpr int R = DP > 128 ? 32 : 64;
  constexpr size_t kv = (2 * (64 + R) * (DP + 4) + 2 * 64 * (R + 4) + 2 * R) * sizeof(float);
  constexpr size_t q = (2 * (64 + R) * (DP + 4) + 64 * (R + 4)) * sizeof(float);
  static_assert(kv <= 227 * 1024, "shared memory");
  cudaError_t e = cudaSuccess;
  if (p.want & 6) {
    const auto k = with_smem(k_attn_any_kv<E, DP, R>, kv);
    e = k ? launch_k(k, p.slots * p.kv_heads, kThreads, kv, s, p) : cudaErrorInvalidValue;
  }
  if (e == cudaSuccess && (p.want & 1)) {
    const auto k = with_smem(k_attn_any_q<E, DP, R>, q);
    e = k ? launch_k(k, p.slots * p.heads, kThreads, q, s, p) : cudaErrorInvalidValue;
  }
  return e;
}

}  // namespace

cudaError_t launch_attn_any_fwd(int es, const AttnPlan& p, cudaStream_t s) {
  if (es == 2)
    return p.dim <= 64 ? any_fwd<__nv_bfloat16, 64>(p, s)
                       : p.dim <= 128 ? any_fwd<__nv_bfloat16, 128>(p, s) : any_fwd<__nv_bfloat16, 256>(p, s);
  return p.dim <= 64 ? any_fwd<float, 64>(p, s)
                     : p.dim <= 128 ? any_fwd<float, 128>(p, s) : any_fwd<float, 256>(p, s);
}

cudaError_t launch_attn_any_bwd(int es, const AttnPlan& p, cudaStream_t s) {
  if (es == 2)
    return p.dim <= 64 ? any_bwd<__nv_bfloat16, 64>(p, s)
                       : p.dim <= 128 ? any_bwd<__nv_bfloat16, 128>(p, s) : any_bwd<__nv_bfloat16, 256>(p, s);
  return p.dim <= 64 ? any_bwd<float, 64>(p, s)
                     : p.dim <= 128 ? any_bwd<float, 128>(p, s) : any_bwd<float, 256>(p, s);
}

cudaError_t launch_attn_rows(int es, const AttnPlan& p, cudaStream_t s) {
  const uint64_t n = uint64_t(p.batch) * p.tokens * p.heads;
  const unsigned cta = unsigned((n + kThreads / 8 * kRowsEach - 1) / (kThreads / 8 * kRowsEach));
  return es == 2 ? launch_k(k_attn_rows<__nv_bfloat16>, cta, kThreads, 0, s, p)
                 : launch_k(k_attn_rows<float>, cta, kThreads, 0, s, p);
}

}  // namespace zr
