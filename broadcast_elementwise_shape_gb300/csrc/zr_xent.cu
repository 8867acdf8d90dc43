// zr_xent.cu — softmax cross entropy of a linear head: small kernels, plan and
// C entry points.  The products are zr_gemm.cuh's.
//
// l[n, v] = x_n . w_v;  lse_n = log sum_v exp(l[n, v]);  the loss of row n with
// label y is lse_n - l[n, y].  The logits are never kept: the forward's product
// reduces each tile to a row's maximum and sum of exponentials in its epilogue
// (8 bytes per row and 128 columns), and the backward computes the logits
// again, a piece of the vocabulary at a time, straight into
//   G[n, v] = c_n (exp(l[n, v] - lse_n) - [v = y]),
// the operand of grad_x = G W and grad_w = G^T X.
//
// bfloat16 tensors are the tensor core's operands as they are.  A binary32
// tensor is split into three bfloat16 parts, x = x0 + x1 + x2 to 2^-24, and a
// product is the sum of the six products of parts whose size reaches 2^-24 of
// the whole: x2 w0 + x1 w1 + x0 w2 + x1 w0 + x0 w1 + x0 w0, each exact in
// binary32 before the accumulation.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "zr_checks.h"
#include "zr_gemm.h"
#include "zr_kernels.cuh"
#include "zr_launch.h"
#include "zr_maps.h"

namespace zr {

// An operand copied into rows the tensor maps can read: [part][row][pitch],
// zero past `cols`.
struct PackPlan {
  const void* in;
  uint16_t* out;
  Decomp rows;               // slot 0
  int64_t inner_stride;
  int64_t part;              // elements between parts
  uint32_t nrow, cols, pitch;
  uint32_t wide;             // 16-byte loads of unit-stride rows
  uint64_t items;            // nrow * pitch / 8; 0: not packed
};

struct XentRows {
  RowLabels labels;
  int64_t ignore_index, vocab;
  uint32_t n;
  int reduction;
  // forward
  const float2* partial;     // [n][slots]
  const float* at;
  uint32_t slots;
  float* lse;
  float* row_loss;           // the losses (no reduction), or workspace: each block's sums
  float* loss;
  uint32_t* ticket;          // blocks done (zeroed by the product before)
  // backward
  const float* grad_loss;
  float* common;             // the factor all rows share (mean, sum)
};

// The backward's first launch: blocks [0, blocks_x) pack x with its left-out
// rows zeroed, the next blocks_w pack w, one more finds the shared factor.
struct PrepPlan {
  PackPlan x, w;
  XentRows rows;
  uint32_t blocks_x, blocks_w, zero_rows;
};

namespace {

template <typename E, int PARTS>
__device__ __forceinline__ void xent_pack(const PackPlan& p, const XentRows* zero, uint64_t i) {
  if (i >= p.items) return;
  const uint32_t nvec = p.pitch / 8;
  const uint32_t row = uint32_t(i / nvec);
  const uint32_t c = uint32_t(i - uint64_t(row) * nvec) * 8;
  float v[8];
  if (zero && row_label(zero->labels, row) == zero->ignore_index) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  } else {
    int64_t off[kMaxOperands];
    decomp_offsets(p.rows, row, off);
    const E* src = static_cast<const E*>(p.in) + off[0] + int64_t(c) * p.inner_stride;
    if (p.wide && c + 8 <= p.cols) {
      if constexpr (sizeof(E) == 4) {
        const float4 lo = reinterpret_cast<const float4*>(src)[0];
        const float4 hi = reinterpret_cast<const float4*>(src)[1];
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
      } else {
        const uint4 q = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < p.cols ? ld1(src + j * p.inner_stride, false) : 0.f;
    }
  }
  uint16_t* dst = p.out + int64_t(row) * p.pitch + c;
#pragma unroll
  for (int part = 0; part < PARTS; ++part, dst += p.part) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
      v[2 * j] -= __uint_as_float(w[j] << 16);
      v[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int T>
__device__ __forceinline__ uint32_t block_count(uint32_t v, uint32_t* s) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) v += s[w];
  return v;
}

template <typename E, int PARTS>
__global__ void __launch_bounds__(kThreads) k_xent_prep(const __grid_constant__ PrepPlan p) {
  pdl_trigger();
  __shared__ uint32_t s_cnt[kThreads / 32];
  uint32_t b = blockIdx.x;
  pdl_wait();
  if (b < p.blocks_x) {
    xent_pack<E, PARTS>(p.x, p.zero_rows ? &p.rows : nullptr, uint64_t(b) * kThreads + threadIdx.x);
    return;
  }
  b -= p.blocks_x;
  if (b < p.blocks_w) {
    xent_pack<E, PARTS>(p.w, nullptr, uint64_t(b) * kThreads + threadIdx.x);
    return;
  }
  const XentRows& r = p.rows;
  if (r.common == nullptr) return;
  uint32_t cnt = 0;
  if (r.reduction == ZR_MEAN) {
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < r.n; i += kThreads) cnt += row_label(r.labels, i) != r.ignore_index;
    cnt = block_count<kThreads>(cnt, s_cnt);
  }
  if (threadIdx.x == 0)
    *r.common = r.reduction == ZR_MEAN ? (cnt ? __fdiv_rn(r.grad_loss[0], float(cnt)) : 0.f)
                                       : r.grad_loss[0];
}

constexpr int kRowsThreads = 256;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// One warp joins a row's partial maxima and sums in a fixed order.  Returns the
// row's loss (0 when it is left out), *used: whether it takes part.
__device__ __forceinline__ float xent_row(const XentRows& p, uint32_t r, uint32_t lane, bool* used) {
  const int64_t y = row_label(p.labels, r);
  const bool known = y >= 0 && y < p.vocab;
  *used = y != p.ignore_index;
  const float at = known ? p.at[r] : __uint_as_float(0x7FFFFFFFu);  // no class: NaN
  const float2* q = p.partial + uint64_t(r) * p.slots;
  // Up to 512 slots stay in registers between the two walks, all loads of a
  // group of 128 in flight together.
  float2 v[4][4];
  float m = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (128 * g >= p.slots) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = lane + 128 * g + 32 * i;
      v[g][i] = k < p.slots ? q[k] : make_float2(-INFINITY, 0.f);
    }
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (128 * g >= p.slots) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, v[g][i].x);
  }
  for (uint32_t i = lane + 512; i < p.slots; i += 32) m = fmaxf(m, q[i].x);
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  // Compensated: beside the slot of a label that is nearly certain, 1, a lane's
  // many others are below its rounding one by one (of 2.1 million classes that
  // lost a thirtieth of 1 - p).
  Kahan s;
  s.init();
  // A slot with no columns has s = 0 and the maximum -inf.
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (128 * g >= p.slots) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.add(__fmul_rn(v[g][i].y, expf(v[g][i].x - base)));
  }
  for (uint32_t i = lane + 512; i < p.slots; i += 32) {
    const float2 w = q[i];
    s.add(__fmul_rn(w.y, expf(w.x - base)));
  }
  const float lse = m + logf(warp_sum(s.s));
  if (lane == 0) p.lse[r] = lse;
  return *used ? lse - at : 0.f;
}

constexpr uint32_t kRowsOneBlock = 32;  // rows that one block joins and totals

// The block's sum of its threads' losses and counts, in thread 0.
__device__ __forceinline__ float block_total(float v, uint32_t* cnt, uint32_t* s_cnt, float* s_sum) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  *cnt = block_count<kRowsThreads>(*cnt, s_cnt);
  return threadIdx.x < 32 ? warp_sum(threadIdx.x < kRowsThreads / 32 ? s_sum[threadIdx.x] : 0.f) : 0.f;
}
__device__ __forceinline__ void write_loss(const XentRows& p, float t, uint32_t cnt) {
  *p.loss = p.reduction == ZR_MEAN ? (cnt ? __fdiv_rn(t, float(cnt)) : 0.f) : t;
}

// ALL: one block joins every row.  Else a warp per row and one sum per block,
// in row_loss as (loss, count); the block that finishes last adds those (which
// one that is changes nothing in the sum).
template <bool ALL>
__global__ void __launch_bounds__(kRowsThreads) k_xent_rows(const __grid_constant__ XentRows p) {
  pdl_trigger();
  __shared__ uint32_t s_cnt[kRowsThreads / 32];
  __shared__ float s_sum[kRowsThreads / 32];
  __shared__ bool s_last;
  const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  Kahan acc;
  acc.init();
  uint32_t cnt = 0;
  const uint32_t step = ALL ? kRowsThreads / 32 : p.n;
  for (uint32_t r = blockIdx.x * (kRowsThreads / 32) + w; r < p.n; r += step) {
    bool used;
    const float loss = xent_row(p, r, lane, &used);
    if (lane == 0) {
      if (p.reduction == ZR_NONE) p.row_loss[r] = loss;
      acc.add(loss);
      cnt += used;
    }
  }
  if (p.reduction == ZR_NONE) return;
  const float t = block_total(acc.s, &cnt, s_cnt, s_sum);
  if constexpr (ALL) {
    if (threadIdx.x == 0) write_loss(p, t, cnt);
  } else {
    float2* sums = reinterpret_cast<float2*>(p.row_loss);
    if (threadIdx.x == 0) {
      sums[blockIdx.x] = make_float2(t, __uint_as_float(cnt));
      __threadfence();
      s_last = atomicAdd(p.ticket, 1u) + 1 == gridDim.x;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    acc.init();
    cnt = 0;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kRowsThreads) {
      const float2 v = __ldcg(sums + i);
      acc.add(v.x);
      cnt += __float_as_uint(v.y);
    }
    const float all = block_total(acc.s, &cnt, s_cnt, s_sum);
    if (threadIdx.x == 0) write_loss(p, all, cnt);
  }
}

// ------------------------------------------------------------------ few rows

// Forward for a few rows of x (generation, scoring): bound by reading w once.
// Each warp takes an equal run of w's rows, two at a time, its lanes 16 bytes
// each, with the next loads in flight while the last are used; x waits in
// shared memory as binary32, and so does the arithmetic run on either storage,
// two columns to an instruction.  The 2 NT sums of two rows of w and NT of x
// are added across the warp by halving: each step exchanges half of what is
// left, until every lane holds one sum (9 exchanges for 8 sums; 40 one by one),
// of which it keeps the running maximum and sum of exponentials.  A block joins
// its warps' in order.  More rows than NT: groups of them, in neighbouring
// blocks, so that L2 serves w to all but one.
//   [50001, 768] bf16: one row 18.5 us with w from DRAM, two 20; the tensor-core
//   path, whose 128-row blocks of x are padding but for the rows, 22.
//   [50001, 768] f32: one row 30 us, 8 rows 42, 16 rows 69; the tensor-core path,
//   which writes w's three parts first, 141.  [32000, 4096] f32: 16 rows 353 us
//   against 434, 24 rows (in three groups) 491.
struct FewPlan {
  const void* x;             // packed or as given: rows of pitch xp
  const void* w;
  int64_t xp, wp;
  uint32_t n, vocab, dim;
  uint32_t groups, slots;    // of NT rows; blocks of each
  RowLabels labels;
  float2* partial;           // [n][slots]
  float* at;
};
constexpr uint32_t kFewElems = 49152;   // rows of x times columns in shared memory, as binary32
constexpr int few_blocks(int rows) { return rows > 1 ? 2 : 3; }  // CTAs per SM
// Rows of x that take this path, and how many of them a block does.
uint32_t few_rows(int es) { return es == 4 ? 16 : 4; }
uint32_t few_nt(uint32_t n) { return n <= 2 ? n : (n <= 4 ? 4 : 8); }

template <typename E, int NT>
__global__ void __launch_bounds__(kThreads, few_blocks(NT))
k_xent_few(const __grid_constant__ FewPlan p) {
  pdl_trigger();
  constexpr int V = 16 / sizeof(E);    // elements per access
  constexpr int R = 2;                 // rows of w at a time
  constexpr int U = 3;                 // accesses per row in flight
  extern __shared__ float s_x[];       // [NT][dim padded to 32 V]
  constexpr int N = R * NT;            // sums: of row i / NT of w and i % NT of x
  constexpr uint32_t kLanes = 32 / N;  // lanes that end up with the same one
  __shared__ float2 s_part[kThreads / 32][N];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t group = blockIdx.x % p.groups, block = blockIdx.x / p.groups;
  const uint32_t t0 = group * NT;
  const uint32_t steps = (p.dim + 32 * V - 1) / (32 * V);
  const uint32_t padded = steps * 32 * V;
  const uint32_t nw = p.slots * (kThreads / 32), me = block * (kThreads / 32) + warp;
  const uint32_t lo = uint32_t(uint64_t(p.vocab) * me / nw);
  const uint32_t hi = uint32_t(uint64_t(p.vocab) * (me + 1) / nw);
  pdl_wait();
  // The position of the next loads: rows v, v + 1, accesses k .. k + U - 1.
  uint32_t lv = lo, lk = 0;
  auto load = [&](uint4 (&q)[U][R]) {
    if (lv >= hi) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const E* row = static_cast<const E*>(p.w) + int64_t(lv + r < hi ? lv + r : lv) * p.wp;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = ((lk + u) * 32 + lane) * V;
        q[u][r] = make_uint4(0, 0, 0, 0);
        if (c + V <= p.dim) {
          q[u][r] = __ldg(reinterpret_cast<const uint4*>(row + c));
        } else if (c < p.dim) {
          alignas(16) E tail[V];  // read as one 16-byte word
#pragma unroll
          for (int j = 0; j < V; ++j) tail[j] = c + j < p.dim ? row[c + j] : E(0.f);
          q[u][r] = *reinterpret_cast<const uint4*>(tail);
        }
      }
    }
    lk += U;
    if (lk >= steps) { lk = 0; lv += R; }
  };
  uint4 qa[U][R], qb[U][R];
  load(qa);
  for (uint32_t i = threadIdx.x; i < NT * padded; i += kThreads) {
    const uint32_t t = i / padded, c = i - t * padded;
    s_x[i] = t0 + t < p.n && c < p.dim
                 ? ld1(static_cast<const E*>(p.x) + int64_t(t0 + t) * p.xp + c, false) : 0.f;
  }
  const uint32_t mine = lane / kLanes, my_r = mine / NT, my_t = t0 + mine % NT;
  int64_t label = -1;
  if (my_t < p.n) label = row_label(p.labels, my_t);
  float m = -INFINITY, s = 0.f;
  __syncthreads();
  F2 acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = f2_splat(0.f);
  uint32_t v = lo, k = 0;
  auto use = [&](const uint4 (&q)[U][R]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u >= steps) break;
      const uint32_t c = ((k + u) * 32 + lane) * V;
      F2 w[R][V / 2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t e[4] = {q[u][r].x, q[u][r].y, q[u][r].z, q[u][r].w};
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          if constexpr (sizeof(E) == 4)
            w[r][j] = f2_pack(__uint_as_float(e[2 * j]), __uint_as_float(e[2 * j + 1]));
          else
            w[r][j] = f2_pack(__uint_as_float(e[j] << 16), __uint_as_float(e[j] & 0xFFFF0000u));
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < V / 2; j += 2) {
          const float4 f = *reinterpret_cast<const float4*>(&s_x[t * padded + c + 2 * j]);
          const F2 x0 = f2_pack(f.x, f.y), x1 = f2_pack(f.z, f.w);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            acc[r * NT + t] = f2_fma(w[r][j], x0, acc[r * NT + t]);
            acc[r * NT + t] = f2_fma(w[r][j + 1], x1, acc[r * NT + t]);
          }
        }
      }
    }
    k += U;
    if (k < steps) return;
    // The rows are complete.
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float hi2;
      f2_unpack(acc[i], a[i], hi2);
      a[i] += hi2;
      acc[i] = f2_splat(0.f);
    }
    uint32_t bit = 16;
#pragma unroll
    for (int h = N / 2; h > 0; h /= 2, bit /= 2) {
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < h; ++i)
        a[i] = (up ? a[i + h] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + h], bit);
    }
#pragma unroll
    for (uint32_t o = kLanes / 2; o > 0; o /= 2) a[0] += __shfl_xor_sync(0xFFFFFFFFu, a[0], o);
    if (v + my_r < hi) {
      const float l = a[0], top = fmaxf(m, l);
      if (lane % kLanes == 0 && int64_t(v + my_r) == label) p.at[my_t] = l;
      const float base = top == -INFINITY ? 0.f : top;
      s = __fmaf_rn(s, __expf(m - base), __expf(l - base));
      m = top;
    }
    k = 0;
    v += R;
  };
  while (v < hi) {
    load(qb);
    use(qa);
    if (v >= hi) break;
    load(qa);
    use(qb);
  }
  if (lane % kLanes == 0) s_part[warp][mine] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x < NT && t0 + threadIdx.x < p.n) {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
      for (int r = 0; r < R; ++r) top = fmaxf(top, s_part[w][r * NT + threadIdx.x].x);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 e = s_part[w][r * NT + threadIdx.x];
        sum = __fmaf_rn(e.y, expf(e.x - base), sum);
      }
    p.partial[uint64_t(t0 + threadIdx.x) * p.slots + block] = make_float2(top, sum);
  }
}

// ------------------------------------------------------------------ plan

// Workspace regions start 256-byte aligned.
size_t take(size_t* at, size_t bytes) {
  const size_t o = *at;
  *at = (o + bytes + 255) / 256 * 256;
  return o;
}

// A matrix operand as the products read it.
struct Operand {
  TDesc t;
  int64_t rows = 0, cols = 0;
  bool one_step = false;     // unit stride along a row, one stride between rows
  int64_t row_step = 0;
  bool pack = false;
  int64_t pitch = 0;         // elements between rows, once packed or as given
  size_t ws = 0;             // offset of the packed copy
  PackPlan pp;
};

// out = scale * the sum of its planes, in their order: results whose k was cut
// into slices (plan_slices).  One pass over planes that are still in L2; four
// columns per thread.
struct JoinPart {
  const float* acc;          // [slices][rows][lda]
  int64_t plane;
  uint32_t slices, rows, cols, vec;
  FastDiv quads;             // lda / 4
  void* out;                 // [rows][cols]
  uint32_t blocks;
};
struct JoinPlan {
  JoinPart p[2];             // of grad_x, grad_w
  const float* scale;        // or null (1)
  XentRows rows;             // left-out rows of part 0 become 0 whatever the factor is
};

__device__ __forceinline__ uint32_t join_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename E>
__global__ void __launch_bounds__(kThreads) k_xent_join(const __grid_constant__ JoinPlan p) {
  pdl_trigger();
  const bool second = blockIdx.x >= p.p[0].blocks;
  const JoinPart& q = second ? p.p[1] : p.p[0];
  const uint32_t i = (blockIdx.x - (second ? p.p[0].blocks : 0u)) * kThreads + threadIdx.x;
  const uint32_t row = fd_div(q.quads, i), c = (i - row * q.quads.d) * 4;
  if (row >= q.rows) return;
  const float* a = q.acc + uint64_t(i) * 4;
  pdl_wait();
  const float scale = p.scale ? *p.scale : 1.f;
  const bool left_out = !second && row_label(p.rows.labels, row) == p.rows.ignore_index;
  float4 v = *reinterpret_cast<const float4*>(a);
#pragma unroll 4
  for (uint32_t k = 1; k < q.slices; ++k) {
    const float4 o = *reinterpret_cast<const float4*>(a + k * q.plane);
    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
  }
  float r[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
  if (left_out) r[0] = r[1] = r[2] = r[3] = 0.f;
  E* out = static_cast<E*>(q.out) + uint64_t(row) * q.cols + c;
  if (q.vec) {
    if constexpr (sizeof(E) == 4) {
      *reinterpret_cast<float4*>(out) = make_float4(r[0], r[1], r[2], r[3]);
    } else {
      *reinterpret_cast<uint2*>(out) = make_uint2(join_bf16(r[0], r[1]), join_bf16(r[2], r[3]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < q.cols) st1(out + j, r[j]);
  }
}

// The label's element of G from the sums that kEpiGrad left (EpiGrad), a warp
// per row, the slots in an order fixed by the sizes.  It goes into G, or, where G
// comes in pieces and the sum is known when the label's piece is long gone, to
// label_g, from which k_xent_spread adds what it contributes.
struct LabelPlan {
  XentRows rows;
  const float* sums;         // [n][slots]
  const float* at;           // [n] exp(l - lse) at the label
  const float* row_scale;    // or null (1)
  uint16_t* g;               // [parts][n][ldg]
  int64_t ldg;
  uint32_t slots, parts;
  float* label_g;            // [n] the sum over the pieces so far, after the last one the element; or null
  uint32_t first, last;
};

__global__ void __launch_bounds__(kRowsThreads) k_xent_label(const __grid_constant__ LabelPlan p) {
  pdl_trigger();
  const uint32_t lane = threadIdx.x & 31, r = blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  if (r >= p.rows.n) return;
  const int64_t y = row_label(p.rows.labels, r);
  // Left out: zeros.  No class: the row is NaN.
  if (y == p.rows.ignore_index || y < 0 || y >= p.rows.vocab) return;
  const float* q = p.sums + uint64_t(r) * p.slots;
  float s = 0.f;
#pragma unroll 4
  for (uint32_t i = lane; i < p.slots; i += 32) s += q[i];
  s = warp_sum(s);
  if (lane != 0) return;
  if (p.label_g && !p.first) s += p.label_g[r];
  if (p.label_g && !p.last) {
    p.label_g[r] = s;
    return;
  }
  float v = -__fdiv_rn(s, s + p.at[r]);
  if (p.row_scale) v *= p.row_scale[r];
  if (p.label_g) {
    p.label_g[r] = v;
    return;
  }
  uint16_t* g = p.g + int64_t(r) * p.ldg + y;
  for (uint32_t part = 0; part < p.parts; ++part, g += int64_t(p.rows.n) * p.ldg) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    *g = *reinterpret_cast<const uint16_t*>(&h);
    v -= __bfloat162float(h);
  }
}

// What the labels' elements add to binary32 gradients whose G came in pieces:
//   grad_x[n] += c g_n w[y_n],   grad_w[v] += c sum over y_n = v of g_n x_n.
// The first blocks take a row of grad_x per warp.  The others take kSpreadClasses
// rows of grad_w and 256 columns each: a block walks all labels, adds the rows
// that are its classes' in their order (no atomics) to shared memory, a column
// per thread, and then to grad_w.  Labels are read V / 32 D / 256 times, from
// L2, and the rest is N D reads and updates, beside 48 N V D operations: [16384,
// 384] x [20000, 384], backward, 3757 us, 3566 of them without the labels'
// elements; 4418 with a pass before the pieces that sums them.
constexpr uint32_t kSpreadClasses = 32;
struct SpreadPlan {
  XentRows rows;
  const float* label_g;
  PackPlan x;                // its layout
  const float* w;
  int64_t w_stride[2];
  float* grad_x;             // or null
  float* grad_w;             // or null
  uint32_t dim, blocks_x, col_blocks;
};

__device__ __forceinline__ bool spread_label(const SpreadPlan& p, int64_t y) {
  return y != p.rows.ignore_index && y >= 0 && y < p.rows.vocab;
}
__global__ void __launch_bounds__(kRowsThreads) k_xent_spread(const __grid_constant__ SpreadPlan p) {
  pdl_trigger();
  __shared__ float s_acc[kSpreadClasses][kRowsThreads];
  __shared__ uint32_t s_row[kRowsThreads], s_class[kRowsThreads], s_cnt[kRowsThreads / 32];
  __shared__ float s_g[kRowsThreads];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  const float common = p.rows.common ? *p.rows.common : 1.f;
  if (blockIdx.x < p.blocks_x) {
    const uint32_t r = blockIdx.x * (kRowsThreads / 32) + warp;
    if (r >= p.rows.n) return;
    const int64_t y = row_label(p.rows.labels, r);
    if (!spread_label(p, y)) return;
    const float f = common * p.label_g[r];
    const float* w = p.w + y * p.w_stride[0];
    float* o = p.grad_x + uint64_t(r) * p.dim;
#pragma unroll 4
    for (uint32_t c = lane; c < p.dim; c += 32) o[c] = __fmaf_rn(f, w[int64_t(c) * p.w_stride[1]], o[c]);
    return;
  }
  const uint32_t b = blockIdx.x - p.blocks_x;
  const int64_t v0 = int64_t(b / p.col_blocks) * kSpreadClasses;
  const uint32_t col = b % p.col_blocks * kRowsThreads + tid;
#pragma unroll
  for (uint32_t k = 0; k < kSpreadClasses; ++k) s_acc[k][tid] = 0.f;
  const float* x = static_cast<const float*>(p.x.in) + (col < p.dim ? int64_t(col) * p.x.inner_stride : 0);
  uint32_t used = 0;         // classes that a row had
  constexpr uint32_t kAhead = 4;
  for (uint32_t r0 = 0; r0 < p.rows.n; r0 += kAhead * kRowsThreads) {
    uint32_t cls[kAhead];
    bool any = false;
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j) {
      const uint32_t r = r0 + j * kRowsThreads + tid;
      const int64_t y = r < p.rows.n ? row_label(p.rows.labels, r) : int64_t(-1);
      const bool in = r < p.rows.n && spread_label(p, y) && y >= v0 && y < v0 + kSpreadClasses;
      cls[j] = in ? uint32_t(y - v0) : kSpreadClasses;
      any |= in;
    }
    if (!__syncthreads_or(any)) continue;
#pragma unroll 1
    for (uint32_t j = 0; j < kAhead; ++j) {
      const bool in = cls[j] < kSpreadClasses;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
      if (lane == 0) s_cnt[warp] = __popc(mask);
      __syncthreads();
      uint32_t at = 0, n = 0;
#pragma unroll
      for (uint32_t k = 0; k < kRowsThreads / 32; ++k) {
        if (k < warp) at += s_cnt[k];
        n += s_cnt[k];
      }
      at += __popc(mask & ((1u << lane) - 1));
      if (in) {
        const uint32_t r = r0 + j * kRowsThreads + tid;
        s_row[at] = r;
        s_class[at] = cls[j];
        s_g[at] = p.label_g[r];
      }
      __syncthreads();
      for (uint32_t i = 0; i < n; i += 4) {
        float xv[4];
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) {
          int64_t off[kMaxOperands] = {};
          if (i + u < n) decomp_offsets(p.x.rows, s_row[i + u], off);
          xv[u] = i + u < n && col < p.dim ? x[off[0]] : 0.f;
        }
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) {
          if (i + u >= n) break;
          const uint32_t k = s_class[i + u];
          s_acc[k][tid] = __fmaf_rn(s_g[i + u], xv[u], s_acc[k][tid]);
          used |= 1u << k;
        }
      }
      __syncthreads();
    }
  }
  if (col >= p.dim) return;
  for (uint32_t m = used; m; m &= m - 1) {
    const uint32_t k = __ffs(m) - 1;
    float* o = p.grad_w + uint64_t(v0 + k) * p.dim + col;
    *o = __fmaf_rn(common, s_acc[k][tid], *o);
  }
}

// Rows up to which the bfloat16 backward holds G in two parts (to 2^-16) rather
// than in one (2^-8): one row block, whose calls wait for w and for launches
// rather than for the tensor cores.  One part shows beside the rounding of the
// result, most of all where few rows leave nothing to average: relative errors
// of the gradients are 0.0026 of [1, 512] x [5000, 512], 0.0019 to 0.0021 of 16
// rows and more; 0.0016 to 0.0017, the result's own rounding, with two.
// Backward, us, one part and two:
//   [50001, 768]:  1 row 68, 78; 128 rows 78, 98; 256 rows 86, 118; 1024 rows 165, 268
//   [32000, 1024]: 16 rows 57, 68; 128 rows 64, 84; 512 rows 89, 133; 4096 rows 444, 763
//   [5000, 512]:   1 row 24, 30; 128 rows 29, 35; 4096 rows 61, 97
constexpr int64_t kTwoPartRows = 128;
constexpr uint64_t kPieceBytes = uint64_t(1) << 30;  // G of one piece of the vocabulary, about

struct XentSet {
  int es = 4;
  uint32_t parts = 1, g_parts = 1;  // of the operands, of G
  bool empty = false;        // no rows
  bool few = false;          // forward by k_xent_few
  Operand x, w;
  TDesc labels;
  XentRows rows;
  size_t ws = 0;
  // forward
  size_t ws_partial = 0, ws_at = 0, ws_row = 0, ws_ticket = 0;
  // backward
  size_t ws_common = 0, ws_g = 0, ws_acc[2] = {0, 0};
  // The label's element: 0 exp(l - lse) - 1; from the rows' sums 1 into G, 2 added
  // to the gradients at the end (LabelPlan).
  int label_pass = 0;
  size_t ws_sums = 0, ws_label = 0;
  int64_t piece = 0, n_piece = 0;
  uint32_t slices[2] = {1, 1};  // of grad_x's and grad_w's k (plan_slices)
};

// CTAs per cluster: pairs when there is more than one CTA's rows.
int pick_cg(int64_t m) { return m > 128 ? 2 : 1; }
// Widest tile (zr_gemm.cuh: a single CTA's stage of three parts).
uint32_t widest(const XentSet& S, int cg) { return S.parts == 3 && cg == 1 ? 128 : 256; }

// Blocks of each group of rows: those of all groups run at the same time.
uint32_t few_slots(int64_t rows, int64_t vocab) {
  const int64_t nt = few_nt(uint32_t(rows)), groups = (rows + nt - 1) / nt;
  return uint32_t(std::min<int64_t>(kSms * few_blocks(int(rows)) / groups, (vocab + 15) / 16));
}

int plan_operand(Operand* o, int es, bool force) {
  const int n = o->t.nd;
  o->cols = o->t.size[n - 1];
  o->rows = 1;
  for (int d = 0; d < n - 1; ++d) o->rows *= o->t.size[d];
  int64_t st[kProbSlots][kMaxDims] = {};
  for (int d = 0; d < n - 1; ++d) st[0][d] = o->t.stride[d];
  Prob P;
  const int rc = coalesce(n - 1, o->t.size, st, 1u, -1, &P);
  if (rc) return rc;
  const int64_t inner = o->cols == 1 ? 1 : o->t.stride[n - 1];
  const bool one = P.n == 1;
  const int64_t pitch = P.st[0][P.n - 1];
  o->one_step = one && inner == 1;
  o->row_step = pitch;
  o->pack = force || es == 4 || !one || inner != 1 || (o->rows > 1 && pitch < o->cols) ||
            pitch % 8 != 0 || o->cols % 64 != 0 ||
            reinterpret_cast<uintptr_t>(o->t.ptr) % 16 != 0;
  o->pitch = (o->cols + 63) / 64 * 64;
  if (!o->pack) {
    if (o->rows > 1) o->pitch = pitch;
    return ZR_OK;
  }
  PackPlan& p = o->pp;
  p = PackPlan{};
  p.in = o->t.ptr;
  p.rows.n = P.n;
  for (int i = 0; i < P.n; ++i) {
    const int d = P.n - 1 - i;
    p.rows.div[i] = make_fastdiv(uint32_t(P.size[d]));
    p.rows.stride[0][i] = P.st[0][d];
  }
  p.inner_stride = inner;
  p.nrow = uint32_t(o->rows);
  p.cols = uint32_t(o->cols);
  p.pitch = uint32_t(o->pitch);
  p.wide = inner == 1 && reinterpret_cast<uintptr_t>(o->t.ptr) % 16 == 0;
  for (int i = 0; i < P.n; ++i)
    if (p.rows.stride[0][i] * es % 16 != 0) p.wide = 0;
  p.part = o->rows * o->pitch;
  p.items = uint64_t(o->rows) * uint64_t(o->pitch / 8);
  return ZR_OK;
}

// Few rows or a small vocabulary leave one gradient with few tiles of long k,
// each longer than an even share of all the work, and the other workers wait
// for them.  Such a gradient's k is cut into slices of about a share (half a
// share for grad_w, whose tiles come last), summed by k_xent_join, where that
// saves more than the join costs.  The last slices end half a slice apart.
//   [40, 384] x [100000, 384] f32, backward: 2258 us whole, 293 in 16 slices;
//   [300, 1024] x [32000, 1024] bf16: 171 us whole, 81 in 4;
//   [16384, 1024] x [500, 1024] bf16, grad_w: 117 us whole, 71 in 7;
//   but [4080, 384] x [5003, 384] f32: 237 us whole, 291 in 2, and
//   [2048, 2048] x [8192, 2048] bf16: 122 us whole, 144 in 2.
// From the sizes alone, whichever gradients a call asks for: a workspace that
// serves both serves one.
void plan_slices(XentSet* S, int64_t dim) {
  const int64_t rows = S->x.rows, n = std::min(S->piece, S->w.rows);
  const int cg = pick_cg(std::min(rows, n));
  const int64_t m[2] = {rows, n}, k[2] = {n, rows};
  const double W = kSms / cg;
  const double us = S->es == 4 ? 2.0 : 0.33;        // a block of k takes
  const double tile_cost = S->es == 4 ? 4 : 6;      // what a tile takes besides, in blocks
  const int64_t least = S->es == 4 ? 2 : 16;        // blocks of a slice
  const int64_t nt = (dim + widest(*S, cg) - 1) / widest(*S, cg);
  double share = 0;
  for (int i = 0; i < 2; ++i)
    share += double((m[i] + 128 * cg - 1) / (128 * cg) * nt) * (double(k[i] + 63) / 64 + tile_cost) / W;
  for (int i = 0; i < 2; ++i) {
    const int64_t kb = (k[i] + 63) / 64;
    const double plane = double(m[i]) * double((dim + 3) / 4 * 4) * 4;
    int64_t len = std::max<int64_t>(int64_t(i ? share / 2 : share), least);
    // All planes together stay within the bound of a piece.
    len = std::max<int64_t>(len, int64_t(double(kb) * plane / double(kPieceBytes)) + 1);
    if (len >= kb) continue;
    const int64_t s = (kb + len - 1) / len, even = (kb + s - 1) / s;
    // A launch, and the planes out and in at 3 TB/s.
    const double join = 8 + 2 * plane * double(s) / 3e6;
    if ((double(kb) - share - double(len) / 2) * us > join)
      S->slices[i] = uint32_t((kb + even - 1) / even);
  }
}

int plan_xent(zr_dtype dtype, const zr_tensor& x, const zr_tensor& w, zr_index it,
              const zr_tensor& labels, int64_t ignore, zr_reduction red, bool back, bool want_w,
              XentSet* S) {
  if (dtype != ZR_F32 && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  if (it != ZR_I32 && it != ZR_I64) return ZR_ERR_DTYPE;
  if (red != ZR_NONE && red != ZR_MEAN && red != ZR_SUM) return ZR_ERR_NULL;
  S->es = dtype == ZR_BF16 ? 2 : 4;
  S->parts = S->es == 4 ? 3 : 1;
  int rc = read_tensor(x, &S->x.t);
  if (rc) return rc;
  if ((rc = read_tensor(w, &S->w.t))) return rc;
  if ((rc = read_tensor(labels, &S->labels))) return rc;
  const int n = S->x.t.nd;
  if (n < 1) return ZR_ERR_RANK;
  if (S->w.t.nd != 2) return ZR_ERR_RANK;
  const int64_t dim = S->x.t.size[n - 1], vocab = S->w.t.size[0];
  if (dim < 1 || vocab < 1 || S->w.t.size[1] != dim) return ZR_ERR_SHAPE;
  if (S->labels.nd != n - 1) return ZR_ERR_SHAPE;
  for (int d = 0; d < n - 1; ++d)
    if (S->labels.size[d] != S->x.t.size[d]) return ZR_ERR_SHAPE;
  // Coordinates, labels and tile counts are 32-bit.
  if (dim >= (int64_t(1) << 24) || vocab >= (int64_t(1) << 30)) return ZR_ERR_SIZE;
  if (S->x.t.numel / dim >= (int64_t(1) << 30)) return ZR_ERR_SIZE;
  if ((S->x.t.numel / dim / 128 + 1) * (vocab / 256 + 1) >= (int64_t(1) << 31)) return ZR_ERR_SIZE;
  if (S->x.t.numel == 0) {
    S->empty = true;
    return ZR_OK;
  }
  if (!S->x.t.ptr || !S->w.t.ptr || !S->labels.ptr) return ZR_ERR_NULL;
  // The backward reads x with the left-out rows zeroed (what they hold must
  // not reach grad_w), so it always copies x: 1 / vocab of the products' work.
  if ((rc = plan_operand(&S->x, S->es, back && want_w))) return rc;
  if ((rc = plan_operand(&S->w, S->es, false))) return rc;
  if (!back && S->x.rows <= few_rows(S->es) &&
      dim * few_nt(uint32_t(S->x.rows)) <= kFewElems) {
    // Rows of elements side by side, w's starting at 16-byte boundaries.
    const int V = 16 / S->es;
    const TDesc& wt = S->w.t;
    S->few = S->x.one_step && (dim == 1 || wt.stride[1] == 1) &&
             (vocab == 1 || wt.stride[0] % V == 0) && reinterpret_cast<uintptr_t>(wt.ptr) % 16 == 0;
    // Three or four bfloat16 rows against much of w that the tensor cores can
    // read as it is: [50001, 768], 29 us here and 22 there; [8000, 512], 8 and 10.
    if (S->es == 2 && S->x.rows > 2 && !S->w.pack && vocab * dim > (int64_t(1) << 24)) S->few = false;
    if (S->few) S->x.pack = S->w.pack = false;
  }
  XentRows& r = S->rows;
  r = XentRows{};
  {
    int64_t st[kProbSlots][kMaxDims] = {};
    for (int d = 0; d < n - 1; ++d) st[0][d] = S->labels.stride[d];
    Prob P;
    if ((rc = coalesce(n - 1, S->labels.size, st, 1u, -1, &P))) return rc;
    // Pitched (a slice of a longer row of labels) and expanded dims, in order.
    for (int d = 0; d + 1 < P.n; ++d)
      if (P.st[0][d] != 0 && P.st[0][d] < P.st[0][d + 1] * P.size[d + 1]) return ZR_ERR_LAYOUT;
    r.labels.n = uint32_t(P.n);
    for (int i = 0; i < P.n; ++i) {
      r.labels.div[i] = make_fastdiv(uint32_t(P.size[P.n - 1 - i]));
      r.labels.stride[i] = P.st[0][P.n - 1 - i];
    }
  }
  r.labels.p = S->labels.ptr;
  r.labels.i64 = it == ZR_I64;
  r.ignore_index = ignore;
  r.vocab = vocab;
  r.n = uint32_t(S->x.rows);
  r.reduction = red;

  size_t at = 0;
  const size_t N = size_t(S->x.rows);
  for (Operand* o : {&S->x, &S->w})
    if (o->pack) o->ws = take(&at, size_t(o->rows) * o->pitch * 2 * S->parts);
  if (!back) {
    const int64_t tn = widest(*S, pick_cg(S->x.rows));
    r.slots = S->few ? few_slots(S->x.rows, vocab) : 2 * uint32_t((vocab + tn - 1) / tn);
    S->ws_partial = take(&at, N * r.slots * sizeof(float2));
    S->ws_at = take(&at, N * 4);
    S->ws_row = take(&at, (N + 7) / 8 * 8);  // (float, count) per block of eight rows
    S->ws_ticket = take(&at, 4);
  } else {
    S->g_parts = S->es == 4 ? 3 : (S->x.rows <= kTwoPartRows ? 2 : 1);
    S->ws_common = take(&at, 4);
    const int64_t most = std::max<int64_t>(2048, int64_t(kPieceBytes / (2 * S->g_parts * N)));
    S->n_piece = (vocab + most - 1) / most;
    S->piece = ((vocab + S->n_piece - 1) / S->n_piece + 255) / 256 * 256;
    S->n_piece = (vocab + S->piece - 1) / S->piece;
    const int64_t wide = std::min<int64_t>(S->piece, (vocab + 63) / 64 * 64);
    S->ws_g = take(&at, N * size_t(wide) * 2 * S->g_parts);
    // bfloat16 in several pieces does without: lse's rounding, some 1e-6 of p, is
    // beside the 2^-8 that G itself is rounded by until p is within 5e-4 of 1.
    S->label_pass = S->n_piece == 1 ? 1 : (S->es == 4 ? 2 : 0);
    if (S->label_pass) {
      const int64_t tn = widest(*S, pick_cg(S->x.rows));
      S->ws_sums = take(&at, N * size_t(2 * ((std::min(S->piece, vocab) + tn - 1) / tn)) * sizeof(float));
      S->ws_at = take(&at, N * 4);
      if (S->label_pass == 2) S->ws_label = take(&at, N * 4);
    }
    plan_slices(S, dim);
    const size_t lda = size_t(dim + 3) / 4 * 4;
    if (S->n_piece > 1 || S->slices[0] > 1) S->ws_acc[0] = take(&at, S->slices[0] * N * lda * 4);
    if (S->slices[1] > 1)
      S->ws_acc[1] = take(&at, S->slices[1] * size_t(std::min(S->piece, vocab)) * lda * 4);
  }
  S->ws = at;
  return ZR_OK;
}

// ------------------------------------------------------------------ launches

// Map of an operand [parts][rows][cols] of bfloat16 (zr_gemm.h): rows `pitch`
// elements apart that hold whole blocks of 64 columns, parts `part` apart;
// rows, blocks and parts out of range read as zero.
cudaError_t operand_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch,
                        uint32_t parts, int64_t part, uint32_t box_rows, uint32_t box_blocks) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {64, cuuint64_t(rows), cuuint64_t(cols + 63) / 64, parts};
  const int64_t plane = parts > 1 ? part : (rows * pitch + 7) / 8 * 8;
  const cuuint64_t strides[3] = {cuuint64_t(pitch) * 2, 128, cuuint64_t(plane) * 2};
  const cuuint32_t box[4] = {64, box_rows, box_blocks, parts}, step[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                        box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Map of an output [parts][rows][cols] of `es` bytes per element that tiles of
// 128 bytes x 32 rows are stored to.
cudaError_t output_map(CUtensorMap* m, void* base, int es, int64_t cols, int64_t rows, int64_t pitch,
                       uint32_t parts, int64_t part) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), parts};
  const int64_t plane = (parts > 1 ? part : rows * pitch) * es;
  const cuuint64_t strides[2] = {cuuint64_t(pitch) * es, cuuint64_t(plane + 15) / 16 * 16};
  const cuuint32_t box[3] = {cuuint32_t(128 / es), 32, 1}, step[3] = {1, 1, 1};
  const CUresult r = fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                        base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Packs the operands that need it; r: the backward's row data, or null.
cudaError_t launch_prep(const XentSet& S, const XentRows* r, char* ws, cudaStream_t s) {
  PrepPlan p = {};
  uint64_t blocks[2] = {0, 0};
  const Operand* ops[2] = {&S.x, &S.w};
  PackPlan* packs[2] = {&p.x, &p.w};
  for (int i = 0; i < 2; ++i) {
    if (!ops[i]->pack) continue;
    *packs[i] = ops[i]->pp;
    packs[i]->out = reinterpret_cast<uint16_t*>(ws + ops[i]->ws);
    blocks[i] = (packs[i]->items + kThreads - 1) / kThreads;
  }
  p.blocks_x = uint32_t(blocks[0]);
  p.blocks_w = uint32_t(blocks[1]);
  const bool shared = r && r->common;
  if (r) p.rows = *r;
  p.zero_rows = r != nullptr;
  const uint64_t n = blocks[0] + blocks[1] + (shared ? 1 : 0);
  if (n == 0) return cudaSuccess;
  if (n >= (uint64_t(1) << 31)) return cudaErrorInvalidValue;
  return S.es == 4 ? launch_k(k_xent_prep<float, 3>, unsigned(n), kThreads, 0, s, p)
                   : launch_k(k_xent_prep<__nv_bfloat16, 1>, unsigned(n), kThreads, 0, s, p);
}

const char* operand_base(const Operand& o, const char* ws) {
  return o.pack ? ws + o.ws : reinterpret_cast<const char*>(o.t.ptr);
}

// The grid, and how two problems' tiles are dealt out (GemmWalk).
unsigned gemm_grid(GemmPlan* g, int cg) {
  const uint32_t W = std::min<uint32_t>(g->tiles, kSms / cg);
  g->workers = W;
  g->head = g->n_prob > 1 ? g->tiles0 % W : 0;
  g->extra = g->late_first = 0;
  if (g->head) {
    const uint32_t k0 = g->pr[0].kb_slice, k1 = g->pr[1].kb_slice;
    g->extra = (k0 + k1 / 2) / k1;
    g->late_first = uint64_t(g->extra) * k1 < k0;
  }
  return unsigned(W * cg);
}

// k blocks per accumulation where chunks are added in registers: one for
// binary32 operands (24 instructions; the truncation is that of the last four,
// beside the roundings of the plain sums), 4096 terms for bfloat16 ones.
constexpr uint32_t kChunkF32 = 1, kChunkBf16 = 64;
// Longest k (in blocks) that bfloat16 results accumulate in one go: its
// truncation stays below 2^-14 of the sum, a 64th of their rounding.  In one go
// up to 131072 terms it reached 2^-10, always towards zero, and gained 1 percent
// or less: [16384, 768] x [50001, 768], backward, 2149 us and 2182 us in chunks;
// [1024, 2048] x [128000, 2048] 1062 and 1067; [4096, 1024] x [32000, 1024] 499
// and 503.
constexpr uint32_t kLongK = 128;

// The logits of bfloat16 rows give binary32 results: at most 1024 terms in one
// go, so that only longer rows pay for the registers.  Forward of 4096 rows and
// 20000 classes, us and the loss's error: 1024 columns in one go 89, 4.5e-7 (in
// two 106); in one go and in chunks 1088 columns 95, 4.5e-7
// and 111, 2.3e-7; 1280 columns 110, 6.0e-7 and 119, 3.1e-7; 2048 columns 172,
// 9.0e-7 and 177, 4.6e-7; 4096 columns 336, 1.8e-6 and 340, 3.8e-7.  The
// backward's logits go the same way, for
// exp(l - lse) - 1 of a row that is learnt shows every difference between them
// and those that lse was summed from: rows of 4096 positive terms, l = 20, had
// the label's gradient off by 1.2 times its size at 1 - p = 1.5e-4 when the
// backward added them in one go.  Backward, in one go and in chunks: 1088 columns
// 343 and 397, 2048 585 and 590, 4096 1154 and 1178.
constexpr uint32_t kChunkLse = 16;

bool sum_chunks(const XentSet& S, int epi, GemmPlan* g) {
  const bool logits = epi != kEpiOut;
  const uint32_t most = S.es == 4 ? 0 : (logits ? kChunkLse : kLongK);
  const uint32_t chunk = S.es == 4 ? kChunkF32 : (logits ? kChunkLse : kChunkBf16);
  bool sum = false;
  for (uint32_t i = 0; i < g->n_prob; ++i) sum |= g->pr[i].kb_slice > most;
  for (uint32_t i = 0; i < g->n_prob; ++i) {
    const uint32_t kb = g->pr[i].kb_slice, n = sum ? (kb + chunk - 1) / chunk : 1;
    g->pr[i].chunk = (kb + n - 1) / n;  // of even length
  }
  return sum;
}
cudaError_t launch_product(const XentSet& S, int epi, int cg, GemmPlan* g, cudaStream_t s) {
  const bool sum = sum_chunks(S, epi, g);
  const unsigned grid = gemm_grid(g, cg);
  return launch_gemm(epi, cg, sum, *g, grid, s);
}

// k in at most `slices` parts.
void set_tiles(GemmProblem* q, int cg, uint32_t slices) {
  q->m_tiles = (q->m + 128 * cg - 1) / (128 * cg);
  q->n_tiles = (q->n + q->tn - 1) / q->tn;
  q->n_kb = (q->k + 63) / 64;
  q->kb_slice = (q->n_kb + slices - 1) / slices;
  q->slices = (q->n_kb + q->kb_slice - 1) / q->kb_slice;
}

// Logits of rows of x against `n` rows of w from row v0.
cudaError_t logits_problem(const XentSet& S, const char* ws, int64_t v0, int64_t n, int cg,
                           GemmPlan* g) {
  GemmProblem& q = g->pr[0];
  q.m = uint32_t(S.x.rows);
  q.n = uint32_t(n);
  q.k = uint32_t(S.x.cols);
  q.tn = widest(S, cg);
  q.a_mn = q.b_mn = 0;
  set_tiles(&q, cg, 1);
  cudaError_t e = operand_map(&q.a, operand_base(S.x, ws), S.x.cols, S.x.rows, S.x.pitch, S.parts,
                              S.x.rows * S.x.pitch, 128, 1);
  if (e != cudaSuccess) return e;
  e = operand_map(&q.b, operand_base(S.w, ws) + v0 * S.w.pitch * 2, S.w.cols, n, S.w.pitch, S.parts,
                  S.w.rows * S.w.pitch, q.tn / cg, 1);
  g->n_prob = 1;
  g->parts = S.parts;
  g->tiles0 = g->tiles = q.m_tiles * q.n_tiles;
  g->m_fast = 1;
  return e;
}

template <typename E>
cudaError_t launch_few(const FewPlan& p, cudaStream_t s) {
  const uint32_t nt = few_nt(p.n);
  constexpr uint32_t step = 32 * 16 / sizeof(E);
  const size_t smem = size_t(nt) * ((p.dim + step - 1) / step * step) * 4;
  auto go = [&](auto* k) {
    if (smem > 40 * 1024) {
      const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), 200 * 1024);
      if (e != cudaSuccess) return e;
    }
    return launch_k(k, p.groups * p.slots, kThreads, smem, s, p);
  };
  if (nt == 1) return go(k_xent_few<E, 1>);
  if (nt == 2) return go(k_xent_few<E, 2>);
  if constexpr (sizeof(E) == 4)
    if (nt == 8) return go(k_xent_few<E, 8>);
  return go(k_xent_few<E, 4>);
}

int run_fwd(const XentSet& S, float* loss, float* lse, char* ws, cudaStream_t s) {
  cudaError_t e;
  if (S.few) {
    XentRows r = S.rows;
    FewPlan p = {};
    p.x = S.x.t.ptr;
    p.w = S.w.t.ptr;
    p.xp = S.x.row_step;
    p.wp = S.w.row_step;
    p.n = r.n;
    p.slots = r.slots;
    p.groups = (r.n + few_nt(r.n) - 1) / few_nt(r.n);
    p.vocab = uint32_t(S.w.rows);
    p.dim = uint32_t(S.x.cols);
    p.labels = r.labels;
    p.partial = reinterpret_cast<float2*>(ws + S.ws_partial);
    p.at = reinterpret_cast<float*>(ws + S.ws_at);
    e = S.es == 4 ? launch_few<float>(p, s) : launch_few<__nv_bfloat16>(p, s);
    if (e != cudaSuccess) return cuda_status(e);
    r.partial = p.partial;
    r.at = p.at;
    r.lse = lse;
    r.row_loss = r.reduction == ZR_NONE ? loss : reinterpret_cast<float*>(ws + S.ws_row);
    r.loss = loss;
    return cuda_status(launch_k(k_xent_rows<true>, 1, kRowsThreads, 0, s, r));
  }
  if ((e = launch_prep(S, nullptr, ws, s)) != cudaSuccess) return cuda_status(e);
  const int cg = pick_cg(S.x.rows);
  GemmPlan g = {};
  if ((e = logits_problem(S, ws, 0, S.w.rows, cg, &g)) != cudaSuccess) return cuda_status(e);
  XentRows r = S.rows;
  r.slots = 2 * g.pr[0].n_tiles;
  r.partial = reinterpret_cast<const float2*>(ws + S.ws_partial);
  r.at = reinterpret_cast<const float*>(ws + S.ws_at);
  r.lse = lse;
  r.row_loss = r.reduction == ZR_NONE ? loss : reinterpret_cast<float*>(ws + S.ws_row);
  r.loss = loss;
  g.labels = r.labels;
  g.partial = reinterpret_cast<float2*>(ws + S.ws_partial);
  g.at = reinterpret_cast<float*>(ws + S.ws_at);
  r.ticket = g.ticket = reinterpret_cast<uint32_t*>(ws + S.ws_ticket);
  if ((e = launch_product(S, kEpiLse, cg, &g, s)) != cudaSuccess) return cuda_status(e);
  if (r.n <= kRowsOneBlock)
    return cuda_status(launch_k(k_xent_rows<true>, 1, kRowsThreads, 0, s, r));
  const unsigned blocks = (r.n + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  return cuda_status(launch_k(k_xent_rows<false>, blocks, kRowsThreads, 0, s, r));
}

int run_bwd(const XentSet& S, const float* grad_loss, const float* lse, void* grad_x, void* grad_w,
            char* ws, cudaStream_t s) {
  XentRows r = S.rows;
  r.grad_loss = grad_loss;
  if (r.reduction != ZR_NONE) r.common = reinterpret_cast<float*>(ws + S.ws_common);
  cudaError_t e = launch_prep(S, &r, ws, s);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t N = S.x.rows, D = S.x.cols, V = S.w.rows;
  uint16_t* G = reinterpret_cast<uint16_t*>(ws + S.ws_g);
  float* acc[2] = {reinterpret_cast<float*>(ws + S.ws_acc[0]),
                   reinterpret_cast<float*>(ws + S.ws_acc[1])};
  JoinPlan join = {};
  join.scale = r.common;
  join.rows = r;
  auto join_part = [&](JoinPart* j, const GemmProblem& q, uint32_t slices, bool vec) {
    j->acc = q.acc;
    j->plane = q.plane;
    j->slices = slices;
    j->rows = q.m;
    j->cols = q.n;
    j->vec = vec;
    j->quads = make_fastdiv(uint32_t(q.lda / 4));
    j->out = q.out;
    j->blocks = uint32_t((uint64_t(q.m) * (q.lda / 4) + kThreads - 1) / kThreads);
  };
  const int64_t lda = (D + 3) / 4 * 4;
  const int per16 = 16 / S.es;
  const unsigned row_blocks = unsigned((N + kRowsThreads / 32 - 1) / (kRowsThreads / 32));
  LabelPlan label = {};
  label.rows = r;
  label.sums = reinterpret_cast<const float*>(ws + S.ws_sums);
  label.at = reinterpret_cast<const float*>(ws + S.ws_at);
  label.row_scale = r.reduction == ZR_NONE ? grad_loss : nullptr;
  label.g = G;
  label.parts = S.g_parts;
  if (S.label_pass == 2) label.label_g = reinterpret_cast<float*>(ws + S.ws_label);
  for (int64_t k = 0; k < S.n_piece; ++k) {
    const int64_t v0 = k * S.piece, n = std::min(S.piece, V - v0);
    const int64_t ldg = (n + 63) / 64 * 64;
    int cg = pick_cg(N);
    GemmPlan g = {};
    if (S.label_pass) {
      g.sums = reinterpret_cast<float*>(ws + S.ws_sums);
      g.at = reinterpret_cast<float*>(ws + S.ws_at);
    }
    if ((e = logits_problem(S, ws, v0, n, cg, &g)) != cudaSuccess) return cuda_status(e);
    g.parts = S.g_parts;
    g.lse = lse;
    g.labels = r.labels;
    g.ignore_index = r.ignore_index;
    g.vocab = V;
    g.row_scale = label.row_scale;
    g.label_base = v0;
    if ((e = output_map(&g.pr[0].c, G, 2, ldg, N, ldg, S.g_parts, N * ldg)) != cudaSuccess)
      return cuda_status(e);
    if ((e = launch_product(S, kEpiGrad, cg, &g, s)) != cudaSuccess) return cuda_status(e);
    if (S.label_pass) {
      label.ldg = ldg;
      label.slots = 2 * g.pr[0].n_tiles;
      label.first = k == 0;
      label.last = k + 1 == S.n_piece;
      if ((e = launch_k(k_xent_label, row_blocks, kRowsThreads, 0, s, label)) != cudaSuccess)
        return cuda_status(e);
    }

    cg = pick_cg(std::min(N, n));
    GemmPlan o = {};
    o.parts = S.g_parts;
    o.out_scale = r.common;
    o.labels = r.labels;
    o.ignore_index = r.ignore_index;
    // grad_x += G W: rows of x, k = this piece's vocabulary.
    if (grad_x) {
      GemmProblem& q = o.pr[o.n_prob++];
      q.m = uint32_t(N);
      q.n = uint32_t(D);
      q.k = uint32_t(n);
      q.tn = widest(S, cg);
      q.a_mn = 0;
      q.b_mn = 1;
      set_tiles(&q, cg, S.slices[0]);
      q.out = grad_x;
      q.ldo = D;
      q.by_row = 1;
      q.acc = acc[0];
      q.lda = lda;
      q.plane = N * lda;
      q.acc_in = k > 0;
      q.acc_out = k + 1 < S.n_piece || S.slices[0] > 1;
      const bool vec = D % per16 == 0 && reinterpret_cast<uintptr_t>(grad_x) % 16 == 0;
      q.tma_out = vec && !q.acc_out;
      if (S.slices[0] > 1 && k + 1 == S.n_piece) join_part(&join.p[0], q, S.slices[0], vec);
      if (q.tma_out && (e = output_map(&q.c, grad_x, S.es, D, N, D, 1, 0)) != cudaSuccess)
        return cuda_status(e);
      if ((e = operand_map(&q.a, G, n, N, ldg, S.g_parts, N * ldg, 128, 1)) != cudaSuccess)
        return cuda_status(e);
      if ((e = operand_map(&q.b, operand_base(S.w, ws) + v0 * S.w.pitch * 2, D, n, S.w.pitch, S.parts,
                           S.w.rows * S.w.pitch, 64, q.tn / cg / 64)) != cudaSuccess)
        return cuda_status(e);
    }
    // This piece's rows of grad_w = G^T X: k = the rows of x.
    if (grad_w) {
      GemmProblem& q = o.pr[o.n_prob++];
      q.m = uint32_t(n);
      q.n = uint32_t(D);
      q.k = uint32_t(N);
      q.tn = widest(S, cg);
      q.a_mn = 1;
      q.b_mn = 1;
      set_tiles(&q, cg, S.slices[1]);
      q.out = static_cast<char*>(grad_w) + v0 * D * S.es;
      q.ldo = D;
      q.acc = acc[1];
      q.lda = lda;
      q.plane = int64_t(n) * lda;
      q.acc_out = S.slices[1] > 1;
      const bool vec = D % per16 == 0 && reinterpret_cast<uintptr_t>(q.out) % 16 == 0;
      q.tma_out = vec && !q.acc_out;
      if (q.acc_out) join_part(&join.p[1], q, q.slices, vec);
      if (q.tma_out && (e = output_map(&q.c, q.out, S.es, D, n, D, 1, 0)) != cudaSuccess)
        return cuda_status(e);
      if ((e = operand_map(&q.a, G, n, N, ldg, S.g_parts, N * ldg, 64, 2)) != cudaSuccess)
        return cuda_status(e);
      if ((e = operand_map(&q.b, operand_base(S.x, ws), D, N, S.x.pitch, S.parts,
                           S.x.rows * S.x.pitch, 64, q.tn / cg / 64)) != cudaSuccess)
        return cuda_status(e);
    }
    o.tiles0 = o.pr[0].m_tiles * o.pr[0].n_tiles * o.pr[0].slices;
    o.tiles = o.tiles0 + (o.n_prob > 1 ? o.pr[1].m_tiles * o.pr[1].n_tiles * o.pr[1].slices : 0);
    o.m_fast = 0;
    if ((e = launch_product(S, kEpiOut, cg, &o, s)) != cudaSuccess) return cuda_status(e);
    if (const unsigned blocks = join.p[0].blocks + join.p[1].blocks) {
      e = S.es == 4 ? launch_k(k_xent_join<float>, blocks, kThreads, 0, s, join)
                    : launch_k(k_xent_join<__nv_bfloat16>, blocks, kThreads, 0, s, join);
      if (e != cudaSuccess) return cuda_status(e);
    }
  }
  if (S.label_pass != 2) return ZR_OK;
  SpreadPlan sp = {};
  sp.rows = r;
  sp.label_g = label.label_g;
  sp.x = S.x.pp;
  sp.w = S.w.t.ptr;
  for (int d = 0; d < 2; ++d) sp.w_stride[d] = S.w.t.stride[d];
  sp.grad_x = static_cast<float*>(grad_x);
  sp.grad_w = static_cast<float*>(grad_w);
  sp.dim = uint32_t(D);
  sp.blocks_x = grad_x ? row_blocks : 0;
  sp.col_blocks = uint32_t((D + kRowsThreads - 1) / kRowsThreads);
  const uint64_t blocks =
      sp.blocks_x + (grad_w ? uint64_t((V + kSpreadClasses - 1) / kSpreadClasses) * sp.col_blocks : 0);
  if (blocks >= (uint64_t(1) << 31)) return ZR_ERR_CUDA;
  return cuda_status(launch_k(k_xent_spread, unsigned(blocks), kRowsThreads, 0, s, sp));
}

std::string xent_json(const XentSet& S) {
  return std::string("{\"kernel\":\"") + (S.few ? "xent_few" : "xent") + "\",\"rows\":" + std::to_string(S.x.rows) + ",\"dim\":" +
         std::to_string(S.x.cols) + ",\"vocab\":" + std::to_string(S.w.rows) + ",\"parts\":" +
         std::to_string(S.parts) + ",\"g_parts\":" + std::to_string(S.g_parts) + ",\"pack_x\":" + std::to_string(S.x.pack) + ",\"pack_w\":" +
         std::to_string(S.w.pack) + ",\"piece\":" + std::to_string(S.piece) + ",\"n_piece\":" +
         std::to_string(S.n_piece) + ",\"slices_x\":" + std::to_string(S.slices[0]) +
         ",\"slices_w\":" + std::to_string(S.slices[1]) + ",\"label_pass\":" + std::to_string(S.label_pass) + ",\"ws\":" + std::to_string(S.ws) + "}";
}

int check_all(std::initializer_list<const void*> ps) {
  for (const void* q : ps) {
    if (!q) continue;
    const int rc = check_device_ptr(q);
    if (rc) return rc;
  }
  return ZR_OK;
}

int64_t loss_count(const XentSet& S, int red) {
  return red == ZR_NONE ? S.x.t.numel / S.x.t.size[S.x.t.nd - 1] : 1;
}

// Outputs against inputs, one another and the workspace.
int check_spans(const XentSet& S, std::initializer_list<Span> outs, std::initializer_list<Span> ins,
                const Span& ws) {
  const Span fixed[3] = {span_of(S.x.t.ptr, S.x.t.extent, S.es), span_of(S.w.t.ptr, S.w.t.extent, S.es),
                         span_of(S.labels.ptr, S.labels.extent, S.rows.labels.i64 ? 8 : 4)};
  for (const Span& f : fixed)
    if (overlaps(f, ws)) return ZR_ERR_LAYOUT;
  for (const Span& i : ins)
    if (overlaps(i, ws)) return ZR_ERR_LAYOUT;
  for (const Span& o : outs) {
    if (overlaps(o, ws)) return ZR_ERR_LAYOUT;
    for (const Span& f : fixed)
      if (overlaps(o, f)) return ZR_ERR_LAYOUT;
    for (const Span& i : ins)
      if (overlaps(o, i)) return ZR_ERR_LAYOUT;
    for (const Span& q : outs)
      if (&q != &o && overlaps(o, q)) return ZR_ERR_LAYOUT;
  }
  return ZR_OK;
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" {

int zr_linear_xent_fwd(zr_dtype dtype, zr_tensor x, zr_tensor w, zr_index label_type,
                       zr_tensor labels, int64_t ignore_index, zr_reduction reduction, float* loss,
                       float* lse, void* workspace, size_t* workspace_bytes, zr_stream_t stream) {
  if (!workspace_bytes) return ZR_ERR_NULL;
  XentSet S;
  int rc = plan_xent(dtype, x, w, label_type, labels, ignore_index, reduction, false, false, &S);
  if (rc) return rc;
  const int64_t nl = loss_count(S, reduction);
  if ((nl > 0 && !loss) || (!S.empty && !lse)) return ZR_ERR_NULL;
  if (workspace && (*workspace_bytes < S.ws || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return ZR_ERR_WORKSPACE;
  const Span ws = span_of(workspace, int64_t(S.ws), 1);
  if (!S.empty &&
      (rc = check_spans(S, {span_of(loss, nl), span_of(lse, S.x.rows)}, {}, ws)))
    return rc;
  if (!workspace) {
    *workspace_bytes = S.ws;
    return ZR_OK;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (S.empty) {
    if (nl == 0) return ZR_OK;
    if ((rc = check_all({loss}))) return rc;
    return cuda_status(cudaMemsetAsync(loss, 0, sizeof(float), st));
  }
  trace("zr_linear_xent_fwd", [&] { return xent_json(S); });
  if ((rc = check_all({S.x.t.ptr, S.w.t.ptr, S.labels.ptr, loss, lse, workspace}))) return rc;
  return run_fwd(S, loss, lse, static_cast<char*>(workspace), st);
}

int zr_linear_xent_bwd(zr_dtype dtype, const float* grad_loss, zr_tensor x, zr_tensor w,
                       zr_index label_type, zr_tensor labels, int64_t ignore_index,
                       zr_reduction reduction, const float* lse, void* grad_x, void* grad_w,
                       void* workspace, size_t* workspace_bytes, zr_stream_t stream) {
  if (!workspace_bytes) return ZR_ERR_NULL;
  XentSet S;
  int rc = plan_xent(dtype, x, w, label_type, labels, ignore_index, reduction, true,
                     grad_w != nullptr, &S);
  if (rc) return rc;
  const int64_t nl = loss_count(S, reduction);
  const int64_t dim = S.w.t.size[1], vocab = S.w.t.size[0];
  if (!S.empty && (!grad_loss || !lse)) return ZR_ERR_NULL;
  if (workspace && (*workspace_bytes < S.ws || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return ZR_ERR_WORKSPACE;
  const Span ws = span_of(workspace, int64_t(S.ws), 1);
  if (!S.empty &&
      (rc = check_spans(S, {span_of(grad_x, grad_x ? S.x.rows * dim : 0, S.es),
                            span_of(grad_w, grad_w ? vocab * dim : 0, S.es)},
                        {span_of(grad_loss, nl), span_of(lse, S.x.rows)}, ws)))
    return rc;
  if (!workspace) {
    *workspace_bytes = S.ws;
    return ZR_OK;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (S.empty) {
    if (!grad_w) return ZR_OK;
    if ((rc = check_all({grad_w}))) return rc;
    return cuda_status(cudaMemsetAsync(grad_w, 0, size_t(vocab) * dim * S.es, st));
  }
  if (!grad_x && !grad_w) return ZR_OK;
  trace("zr_linear_xent_bwd", [&] { return xent_json(S); });
  if ((rc = check_all({grad_loss, S.x.t.ptr, S.w.t.ptr, S.labels.ptr, lse, grad_x, grad_w, workspace})))
    return rc;
  return run_bwd(S, grad_loss, lse, grad_x, grad_w, static_cast<char*>(workspace), st);
}

int zr_test_describe_linear_xent(zr_dtype dtype, zr_tensor x, zr_tensor w, zr_index label_type,
                                 zr_tensor labels, int backward, char* buf, size_t len) {
  XentSet S;
  const int rc = plan_xent(dtype, x, w, label_type, labels, -100, ZR_MEAN, backward != 0, backward != 0, &S);
  if (rc) return rc;
  return copy_json(S.empty ? std::string("{\"kernel\":\"none\"}") : xent_json(S), buf, len);
}

int zr_test_gemm_walk(uint32_t tiles0, uint32_t tiles1, uint32_t kb0, uint32_t kb1, int cg,
                      uint32_t* visits, uint64_t* load, uint32_t* workers) {
  if (!visits || !load || !workers || tiles0 == 0 || kb0 == 0 || kb1 == 0 || (cg != 1 && cg != 2))
    return ZR_ERR_NULL;
  GemmPlan g = {};
  g.n_prob = tiles1 ? 2 : 1;
  g.pr[0].kb_slice = kb0;
  g.pr[1].kb_slice = kb1;
  g.tiles0 = tiles0;
  g.tiles = tiles0 + tiles1;
  *workers = gemm_grid(&g, cg) / unsigned(cg);
  for (uint32_t t = 0; t < g.tiles; ++t) visits[t] = 0;
  for (uint32_t w = 0; w < *workers; ++w) {
    GemmWalk k = gemm_walk(g, w);
    load[w] = 0;
    for (uint32_t t; (t = gemm_next(g, &k)) < g.tiles;) {
      ++visits[t];
      load[w] += t < tiles0 ? kb0 : kb1;
    }
  }
  return ZR_OK;
}

}  // extern "C"
