// zr_gemm.cuh — persistent tcgen05 product with fused epilogues (sm_103a).
//
// A tile is 128 rows per CTA by up to 256 columns, k in blocks of 64.  Warp 8
// brings operand blocks by TMA (128-byte swizzle) through a ring in shared
// memory, warp 9 issues the tensor-core instructions, and warps 0-7 run the
// epilogue: 32 rows (TMEM lanes) and half the columns each.  The accumulator
// is double-buffered in TMEM (2 x 256 columns), so one tile's epilogue
// overlaps the next one's products.  With CG = 2 a cluster of two CTAs shares
// a tile of 256 rows: each loads its own 128 rows of A and half of B's
// columns, and the pair's tensor cores read both halves, which cuts the
// operand traffic from L2 by a third.
//
// Every wait has a limit (kWaitNs).  When one runs out, the CTA sets its
// abort flag, all its roles leave their loops, in-flight copies get time to
// land before TMEM is freed, and the epilogue fills the CTA's remaining tiles
// with NaN: a failure shows in the results, nothing hangs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zr_gemm.h"
#include "zr_kernels.cuh"
#include "zr_tc.cuh"

namespace zr {

constexpr int kGemmThreads = 320;      // 8 epilogue warps, producer, issuer
constexpr uint32_t kGemmM = 128;       // rows per CTA
constexpr uint32_t kGemmK = 64;        // k per block (128 bytes)
constexpr uint32_t kABytes = kGemmM * kGemmK * 2;

// Parts of the operands A and B, and the products of parts that make up theirs.
// PARTS = 3 (binary32 tensors): a stage holds all three parts of both operands,
// which its six products share; half the traffic of loading a pair of parts for
// each.  Tiles of a single CTA are then at most 128 columns wide.  (Four stages
// of half the k instead of two: [2048, 1024] x [8192, 1024] f32 backward 434 us
// against 405.)
// PARTS = 2 (bfloat16 tensors, G in two parts): A of the gradients' products.
template <int EPI, int CG, int PARTS>
struct GemmCfg {
  static constexpr uint32_t kA = PARTS == 2 && EPI != kEpiOut ? 1 : PARTS;
  static constexpr uint32_t kB = PARTS == 3 ? 3 : 1;
  static constexpr int kPairs = PARTS == 3 ? 6 : kA;
  static constexpr uint32_t kBBytes = (PARTS == 3 ? 128 : 256 / CG) * kGemmK * 2;
  static constexpr uint32_t kStageBytes = kA * kABytes + kB * kBBytes;
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  // The ring, 4 KB of output staging per epilogue warp, alignment.
  static constexpr uint32_t kOutAt = kStages * kStageBytes;
  static constexpr uint32_t kSmem = kOutAt + 8 * 4096 + 1024;
};

struct GemmTile {
  uint32_t prob, mt, nt, n0, tn;
  uint32_t slice, kb0, n_kb; // its blocks of k
};
template <int EPI, int CG>
__device__ __forceinline__ GemmTile gemm_tile(const GemmPlan& p, uint32_t t) {
  GemmTile g;
  g.prob = t >= p.tiles0 ? 1u : 0u;
  uint32_t l = t - (g.prob ? p.tiles0 : 0u);
  const GemmProblem& q = p.pr[g.prob];
  g.slice = g.kb0 = 0;
  g.n_kb = q.n_kb;
  if (EPI == kEpiOut && q.slices > 1) {
    const uint32_t per = q.m_tiles * q.n_tiles;
    g.slice = l / per;
    l -= g.slice * per;
    g.kb0 = g.slice * q.kb_slice;
    const uint32_t left = q.n_kb - g.kb0;
    g.n_kb = left < q.kb_slice ? left : q.kb_slice;
  }
  if (p.m_fast) {
    g.nt = l / q.m_tiles;
    g.mt = l - g.nt * q.m_tiles;
  } else {
    g.mt = l / q.n_tiles;
    g.nt = l - g.mt * q.n_tiles;
  }
  g.n0 = g.nt * q.tn;
  g.tn = q.tn;
  if (q.b_mn) {  // each CTA's share is whole blocks of 64
    const uint32_t left = (q.n - g.n0 + 64 * CG - 1) / (64 * CG) * (64 * CG);
    if (left < g.tn) g.tn = left;
  }
  return g;
}

// The pairs of parts (a, b) of a block of k in the order they are added:
// smallest products first, so that the sum is small until the last, largest
// pair (parts 0, 0).
template <int PAIRS>
__device__ __forceinline__ constexpr uint32_t gemm_pair(int i, int operand) {
  if (PAIRS < 6) return operand == 0 ? PAIRS - 1 - i : 0;
  constexpr uint32_t pairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
  return pairs[i][operand];
}

// ------------------------------------------------------------------ epilogues

// Where one epilogue warp's lane stands: row `row` (live: inside the product)
// of the warp's 32 from row0, columns c0, c0 + 128, ... of the tile in chunks
// of 64, tile column 0 = column n0.
struct EpiPos {
  uint32_t row, row0, n0, c0, tn, nt, half, slice, lane;
  uint32_t out;              // the warp's 4 KB of staging
  bool live, ok;
};

// 64 bfloat16 columns of the warp's 32 rows to global memory: each lane writes
// its row into the staging (128-byte swizzle), one lane starts the TMA store.
// 16-byte stores straight from the lanes touch 32 rows per instruction, half a
// sector each; the gradient epilogue took 570 us with them on a [16384, 25088]
// piece.
__device__ __forceinline__ void epi_begin_store(const EpiPos& e) {
  // The staging's last store has been read.
  if (e.lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void epi_stage(const EpiPos& e, int i, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(e.out + e.lane * 128 +
                                                               ((i ^ (e.lane & 7)) << 4)),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void epi_end_store(const CUtensorMap* map, const EpiPos& e, uint32_t c,
                                              int part) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (e.lane == 0) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            map),
        "r"(e.out), "r"(int(e.n0 + c)), "r"(int(e.row0)), "r"(part)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void epi_store(const CUtensorMap* map, const EpiPos& e, uint32_t c,
                                          int part, float* v) {
  epi_begin_store(e);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    epi_stage(e, i, pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
              pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  epi_end_store(map, e, c, part);
}
// The same of 32 binary32 columns.  [4080, 384] x [5003, 384] f32, backward:
// 234 us with the lanes' own stores, 228 with these.
__device__ __forceinline__ void epi_store_f32(const CUtensorMap* map, const EpiPos& e, uint32_t c,
                                              const float* v) {
  epi_begin_store(e);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    epi_stage(e, i, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
              __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  epi_end_store(map, e, c, 0);
}

// Running maximum and sum of exponentials over the lane's columns, in one
// walk: a chunk's maximum rescales the sum once.  The maximum (in EpiGrad, lse)
// is subtracted before the factor log2(e): near it, where terms count, that
// difference is exact, while one fused step from the rounded product
// max * log2(e) would put its rounding, 1e-6 at 20, into every term.
struct EpiLse {
  int64_t at;                // column of the label in this tile
  float m, s;

  __device__ __forceinline__ void begin(const GemmPlan& p, const GemmProblem&, const EpiPos& e) {
    const int64_t label = e.live ? row_label(p.labels, e.row) : int64_t(-1);
    at = e.live ? label - int64_t(e.n0) : int64_t(-1);
    m = -INFINITY;
    s = 0.f;
  }
  __device__ __forceinline__ void chunk(const GemmPlan& p, const GemmProblem& q, const EpiPos& e,
                                        uint32_t c, float* v) {
    if (e.n0 + c + 64 > q.n) {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (e.n0 + c + i >= q.n) v[i] = -INFINITY;
    }
    if (__any_sync(0xFFFFFFFFu, at >= int64_t(c) && at < int64_t(c) + 64)) {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (at == int64_t(c) + i) p.at[e.row] = e.ok ? v[i] : qnan();
    }
    float top[4] = {m, v[1], v[2], v[3]};
    top[0] = fmaxf(top[0], v[0]);
#pragma unroll
    for (int i = 4; i < 64; i += 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top[j] = i + 4 + j < 64 ? fmaxf(fmaxf(top[j], v[i + j]), v[i + 4 + j]) : fmaxf(top[j], v[i + j]);
    }
    const float mn = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float base = mn == -INFINITY ? 0.f : mn;
    const F2 k = f2_splat(kLog2e), off = f2_splat(-base);
    F2 add[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) add[i] = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float lo, hi;
      f2_unpack(f2_mul(f2_add(f2_pack(v[2 * i], v[2 * i + 1]), off), k), lo, hi);
      add[i & 3] = f2_add(add[i & 3], f2_pack(ex2(lo), ex2(hi)));
    }
    float lo, hi;
    f2_unpack(f2_add(f2_add(add[0], add[1]), f2_add(add[2], add[3])), lo, hi);
    s = __fmaf_rn(s, ex2((m - base) * kLog2e), lo + hi);
    m = mn;
  }
  __device__ __forceinline__ void end(const GemmPlan& p, const GemmProblem& q, const EpiPos& e) {
    if (e.live)
      p.partial[uint64_t(e.row) * (2 * q.n_tiles) + 2 * e.nt + e.half] =
          e.ok ? make_float2(m, s) : make_float2(0.f, qnan());
  }
};

// G = scale * (exp(l - lse) - [column is the label]).  G is the operand of
// the two gradient products, so it is stored as their operand type: for binary32
// tensors as three bfloat16 parts that hold it to 2^-24, for bfloat16 ones
// rounded once (2^-8 of an element at most) or, for few rows, in two parts.  One
// part's rounding is as large as that of the bfloat16 results and independent of
// it.  A result that averages over many elements shows little of it, but a class
// that is one row's label has that row's G as its main factor however many rows
// there are: over all of a gradient the error grew from 0.0017 of it, the
// results' rounding, to 0.0019 or 0.0020.  A second part costs half of the step
// again where the tensor cores bound it (kTwoPartRows).  A factor that all rows
// share is left to the products' epilogue: then the label's element of a row that
// is not yet learnt, the largest by far, is -1 and rounds to itself.
//
// The label's element, p - 1, is a small difference where the row is learnt:
// lse's rounding alone (2^-25 of it) was 1.7e-5 of a whole binary32 gradient of
// one row.  So it is taken as what the other elements sum to, which is as exact
// as they are: with p.sums every half tile leaves its sum of exp(l - lse) but
// for the label's, and -sum / (sum + the label's) takes its place (k_xent_label).
template <int PARTS>
struct EpiGrad {
  float scale, lse, sum;
  int64_t at;                // column of the label in this tile
  bool out;                  // the row is left out: zeros, whatever its products are

  __device__ __forceinline__ void begin(const GemmPlan& p, const GemmProblem&, const EpiPos& e) {
    scale = 1.f;
    lse = sum = 0.f;
    at = -1;
    out = true;
    if (e.live) {
      const int64_t label = row_label(p.labels, e.row);
      out = label == p.ignore_index;
      if (!out) {
        if (p.row_scale) scale = p.row_scale[e.row];
        lse = p.lse[e.row];
        if (label < 0 || label >= p.vocab) scale = qnan();  // no class: NaN, not a guess
        else at = label - p.label_base - int64_t(e.n0);
      }
    }
  }
  __device__ __forceinline__ void chunk(const GemmPlan& p, const GemmProblem& q, const EpiPos& e,
                                        uint32_t c, float* v) {
    const F2 k = f2_splat(kLog2e), off = f2_splat(-lse);
    float low = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      f2_unpack(f2_mul(f2_add(f2_pack(v[2 * i], v[2 * i + 1]), off), k), v[2 * i], v[2 * i + 1]);
      low = fminf(fminf(low, v[2 * i]), v[2 * i + 1]);
    }
    // The short exponential flushes subnormal results; the gradient of a class
    // that is all but impossible is as exact as any other.
    if (__any_sync(0xFFFFFFFFu, low < -126.f)) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = ex2_full(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = ex2(v[i]);
    }
    // G's rows are padded with zeros to whole blocks of 64.
    const bool ragged = e.n0 + c + 64 > q.n;
    if (ragged) {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (e.n0 + c + i >= q.n) v[i] = 0.f;
    }
    const bool mine = at >= int64_t(c) && at < int64_t(c) + 64;
    if (__any_sync(0xFFFFFFFFu, mine)) {
      if (p.sums) {
        float own = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          if (at == int64_t(c) + i) {
            own = v[i];
            v[i] = 0.f;
          }
        }
        if (mine) p.at[e.row] = e.ok ? own : qnan();
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (at == int64_t(c) + i) v[i] -= 1.f;
      }
    }
    if (p.sums) {
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int i = 0; i < 64; i += 2) { lo += v[i]; hi += v[i + 1]; }
      sum += lo + hi;
    }
    if (__any_sync(0xFFFFFFFFu, scale != 1.f)) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] *= scale;
      if (ragged || (p.sums && mine)) {  // an infinite factor leaves what is no element 0
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (e.n0 + c + i >= q.n || (p.sums && at == int64_t(c) + i)) v[i] = 0.f;
      }
    }
    if (out || !e.ok) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = e.ok ? 0.f : qnan();
    }
    epi_store(&q.c, e, c, 0, v);
    #pragma unroll 1
    for (int part = 1; part < PARTS; ++part) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
      epi_store(&q.c, e, c, part, v);
    }
  }
  __device__ __forceinline__ void end(const GemmPlan& p, const GemmProblem& q, const EpiPos& e) {
    if (p.sums && e.live)
      p.sums[uint64_t(e.row) * (2 * q.n_tiles) + 2 * e.nt + e.half] = e.ok ? sum : qnan();
  }
};

// Results in the operands' type: binary32 where they come in three parts.
template <int PARTS>
struct EpiOut {
  // -0: the row is left out, and an infinite factor makes no NaN of its zeros
  // (a sentinel and not a flag beside it: the tile's values take the registers).
  float scale;

  __device__ __forceinline__ void begin(const GemmPlan& p, const GemmProblem& q, const EpiPos& e) {
    scale = p.out_scale && !q.acc_out ? *p.out_scale : 1.f;
    if (q.by_row && e.live && row_label(p.labels, e.row) == p.ignore_index) scale = -0.f;
  }
  __device__ __forceinline__ void chunk(const GemmPlan& p, const GemmProblem& q, const EpiPos& e,
                                        uint32_t c, float* v) {
    const uint32_t n = e.n0 + c;
    float* acc = q.acc + int64_t(e.slice) * q.plane + int64_t(e.row) * q.lda + n;  // rows of acc are padded to groups of 4
    if (q.acc_in && e.live) {
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        if (n + i < q.n) {
          const float4 o = *reinterpret_cast<const float4*>(acc + i);
          v[i] += o.x; v[i + 1] += o.y; v[i + 2] += o.z; v[i + 3] += o.w;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] *= scale;
    if (__float_as_uint(scale) == 0x80000000u || !e.ok) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = e.ok ? 0.f : qnan();
    }
    if (q.acc_out) {
      if (e.live) {
#pragma unroll
        for (int i = 0; i < 64; i += 4)
          if (n + i < q.n)
            *reinterpret_cast<float4*>(acc + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
      return;
    }
    if (q.tma_out) {
      if constexpr (PARTS != 3) {
        epi_store(&q.c, e, c, 0, v);
      } else {
        epi_store_f32(&q.c, e, c, v);
        if (n + 32 < q.n) epi_store_f32(&q.c, e, c + 32, v + 32);
      }
      return;
    }
    if (!e.live) return;
    if constexpr (PARTS == 3) {
      float* o = static_cast<float*>(q.out) + int64_t(e.row) * q.ldo + n;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (n + i < q.n) o[i] = v[i];
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(q.out) + int64_t(e.row) * q.ldo + n;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (n + i < q.n) o[i] = __float2bfloat16_rn(v[i]);
    }
  }
  __device__ __forceinline__ void end(const GemmPlan&, const GemmProblem&, const EpiPos&) {}
};

template <int EPI, int PARTS>
struct EpiOf { using type = EpiLse; };
template <int PARTS>
struct EpiOf<kEpiGrad, PARTS> { using type = EpiGrad<PARTS>; };
template <int PARTS>
struct EpiOf<kEpiOut, PARTS> { using type = EpiOut<PARTS>; };

// ------------------------------------------------------------------ kernel

// SUM: the accumulator covers only q.chunk blocks of k, and the epilogue warps
// add the chunks in registers, rounding to nearest.  The tensor core's own
// accumulation truncates: sums of positive terms fell short by 1.2 to 1.4 times
// 2^-24 of their size per 16 terms (7.1e-5 at k = 16384), always towards zero.
// Results of 24 bits need the chunks; those of 8 bits do without until k is
// some hundred thousand.
template <int EPI, int CG, bool SUM, int PARTS>
__global__ void __launch_bounds__(kGemmThreads, 1) k_gemm(const __grid_constant__ GemmPlan p) {
  using Cfg = GemmCfg<EPI, CG, PARTS>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_full[S], s_empty[S], s_tfull[2], s_tempty[2];
  __shared__ uint32_t s_tmem, s_abort;
  pdl_trigger();
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : uniform(cluster_rank());
  const uint32_t ring = (smem_u32(s_raw) + 1023u) & ~1023u;
  volatile uint32_t* abort = &s_abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_tfull[i]), 1);
      mbar_init(smem_u32(&s_tempty[i]), 8 * CG);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<CG>(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  GemmWalk walk = gemm_walk(p, blockIdx.x / CG);
  pdl_wait();
  if (EPI == kEpiLse && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;

  if (warp == 8) {
    // Producer: this CTA's rows of A and its share of B's columns.  The whole
    // warp walks and waits, one lane starts the copies (see the issuer).
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (uint32_t t; ok && (t = gemm_next(p, &walk)) < p.tiles;) {
      const GemmTile g = gemm_tile<EPI, CG>(p, t);
      const GemmProblem& q = p.pr[g.prob];
      const uint32_t m0 = (g.mt * CG + rank) * kGemmM;
      const uint32_t n0 = g.n0 + rank * (g.tn / CG);
      // Whole boxes, whatever part of them is inside the operand.
      const uint32_t bytes = (Cfg::kA * kABytes + Cfg::kB * (q.tn / CG * kGemmK * 2)) * CG;
      const uint32_t end = g.kb0 + g.n_kb, a_mn = q.a_mn, b_mn = q.b_mn;
      for (uint32_t kb = g.kb0; kb < end; ++kb) {
        ok = warp_wait(smem_u32(&s_empty[stage]), phase ^ 1, abort);
        if (!ok) break;
        if (leader) {
          const uint32_t local = smem_u32(&s_full[stage]);
          if (rank == 0) mbar_expect(local, bytes);
          const uint32_t bar = CG == 1 ? local : cluster_addr(local, 0);
          const uint32_t sa = ring + stage * Cfg::kStageBytes, sb = sa + Cfg::kA * kABytes;
          tma_load<CG>(sa, &q.a, bar, a_mn ? kb * kGemmK : m0, a_mn ? m0 / 64 : kb);
          tma_load<CG>(sb, &q.b, bar, b_mn ? kb * kGemmK : n0, b_mn ? n0 / 64 : kb);
        }
        __syncwarp();
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
    }
    // Every slot is read before the CTA may end (and its peer's signals are in).
    for (int i = 0; i < S && ok; ++i) {
      ok = warp_wait(smem_u32(&s_empty[stage]), phase ^ 1, abort);
      if (++stage == S) { stage = 0; phase ^= 1; }
    }
  } else if (warp == 9 && rank == 0) {
    // Issuer.  The whole warp walks and waits, one lane issues: control flow and
    // operands are then the same for the warp, and a block of k is a few
    // instructions to the tensor core with little to work out between them.
    // With one lane in the loop the tensor core waited for its instructions:
    // [16384, 768] x [50001, 768], 755 us against 624 us now.
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 0, it = 0;
    bool ok = true;
    for (uint32_t t; ok && (t = gemm_next(p, &walk)) < p.tiles;) {
      const GemmTile g = gemm_tile<EPI, CG>(p, t);
      const GemmProblem& q = p.pr[g.prob];
      // D binary32, A and B bfloat16, their majors, N / 8, M / 16.
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (q.a_mn << 15) | (q.b_mn << 16) |
                             ((g.tn >> 3) << 17) | (uint32_t(kGemmM * CG / 16) << 24);
      const uint32_t ka = q.a_mn ? 2048 >> 4 : 32 >> 4, kb16 = q.b_mn ? 2048 >> 4 : 32 >> 4;
      const uint64_t da = operand_desc(ring, q.a_mn);
      const uint64_t db = operand_desc(ring + Cfg::kA * kABytes, q.b_mn);
      const uint32_t n_kb = g.n_kb, chunk = q.chunk;
      for (uint32_t k1 = 0; k1 < n_kb && ok; k1 += chunk, ++it) {
        const uint32_t buf = it & 1;
        ok = warp_wait(smem_u32(&s_tempty[buf]), ((it >> 1) & 1) ^ 1, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        const uint32_t nk = n_kb - k1 < chunk ? n_kb - k1 : chunk;
        for (uint32_t kb = 0; kb < nk; ++kb) {
          ok = warp_wait(smem_u32(&s_full[stage]), phase, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t at = stage * (Cfg::kStageBytes >> 4);
#pragma unroll
            for (int i = 0; i < Cfg::kPairs; ++i) {
              const uint64_t pa = da + at + gemm_pair<Cfg::kPairs>(i, 0) * (kABytes >> 4);
              const uint64_t pb = db + at + gemm_pair<Cfg::kPairs>(i, 1) * (Cfg::kBBytes >> 4);
#pragma unroll
              for (uint32_t j = 0; j < kGemmK / 16; ++j)
                tc_mma<CG>(d, pa + j * ka, pb + j * kb16, idesc, (kb | i | j) != 0);
            }
            tc_commit<CG>(smem_u32(&s_empty[stage]));
          }
          __syncwarp();
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
        if (ok && leader) tc_commit<CG>(smem_u32(&s_tfull[buf]));
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    uint32_t it = 0;
    bool ok = true;
    const uint32_t quad = warp & 3, half = warp >> 2;
    for (uint32_t t; (t = gemm_next(p, &walk)) < p.tiles;) {
      const GemmTile g = gemm_tile<EPI, CG>(p, t);
      const GemmProblem& q = p.pr[g.prob];
      EpiPos e;
      e.row0 = (g.mt * CG + rank) * kGemmM + quad * 32;
      e.row = e.row0 + lane;
      e.lane = lane;
      e.out = ring + Cfg::kOutAt + warp * 4096;
      e.live = e.row < q.m;
      e.n0 = g.n0;
      e.c0 = half * 64;
      e.tn = g.tn;
      e.nt = g.nt;
      e.half = half;
      e.slice = g.slice;
      typename EpiOf<EPI, PARTS>::type epi;
      epi.begin(p, q, e);
      auto acquire = [&]() {
        const uint32_t buf = it & 1;
        ok = ok && warp_wait(smem_u32(&s_tfull[buf]), (it >> 1) & 1, abort);
        tc_fence_after();
        e.ok = ok;
        return tmem + (quad << 21) + buf * 256;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = smem_u32(&s_tempty[it & 1]);
          mbar_arrive_cluster(CG == 1 ? bar : cluster_addr(bar, 0));
        }
        ++it;
      };
      if constexpr (!SUM) {
        // The tile's values move to registers at once, so that the tensor core
        // gets its accumulator back before they are worked on.
        const uint32_t d = acquire();
        float v[2][64];
        __syncwarp();
        if (e.c0 < e.tn) tc_load64(d + e.c0, v[0]);
        if (e.c0 + 128 < e.tn) tc_load64(d + e.c0 + 128, v[1]);
        release();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t c = e.c0 + j * 128;
          __syncwarp();
          if (c < e.tn && e.n0 + c < q.n) epi.chunk(p, q, e, c, v[j]);
        }
      } else {
        float v[2][64];
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i / 64][i % 64] = 0.f;
        for (uint32_t k1 = 0; k1 < g.n_kb; k1 += q.chunk) {
          const uint32_t d = acquire();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t c = e.c0 + (j / 2) * 128 + (j & 1) * 32;
            if (c < e.tn) {
              float w[32];
              __syncwarp();
              tc_load32(d + c, w);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[j / 2][(j & 1) * 32 + i] += w[i];
            }
          }
          release();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t c = e.c0 + j * 128;
          __syncwarp();
          if (c < e.tn && e.n0 + c < q.n) epi.chunk(p, q, e, c, v[j]);
        }
      }
      epi.end(p, q, e);
    }
    // This warp's stores are complete.
    if (EPI != kEpiLse && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if (*abort) {
    // Copies and products still in flight land within this time.
    const uint64_t t0 = timer_ns();
    while (timer_ns() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free<CG>(tmem, 512);
}

}  // namespace zr
