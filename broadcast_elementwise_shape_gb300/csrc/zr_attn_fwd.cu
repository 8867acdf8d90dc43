// zr_attn_fwd.cu — causal attention, forward, on the tensor cores.
//
// A CTA works on two tiles of 128 queries of a head, which share the keys and
// values that go past: warp 8 brings them by TMA, warp 9 issues the products,
// and the warps 0-3 and 4-7 each turn the scores of their tile into weights, one
// row per thread, while the tensor core works for the other tile.  Scores,
// weights and the running result stay in tensor memory: S (128 columns,
// binary32) is read once, the weights are written over it as bfloat16, the A
// operand of the product with the values.  When a row's maximum grows, the warp
// rescales its result in tensor memory: the products before are complete by
// then, since the scores that follow them are.  The maximum is always the row's
// own, so that the weight of a token that has it is 1 without rounding, and a
// row whose weight is nearly all on one token is exact where it must be.
//
// [2, 8192] tokens of 16 heads of 128: 367 us, 1.5 PFLOP/s of the pairs that see
// one another; of 12 heads of 64: 214 us, 0.97.  Heads of 64 are bound by the
// warps' round from one tile's scores to the next's (issue slots 41 % busy, the exponential
// unit 31 %, the tensor pipe 30 to 35 %).  What did not help there is in the
// order of the tensor core's work: scores ahead of the weights (weights in columns of their
// own, 214 -> 246 us: the two tiles' warps then wait together instead of in turn), a
// quarter of the exponentials as polynomials on the multiply-add units (240).
//
// CTAs are persistent, one per SM; the tiles are dealt out heaviest first, there
// and back.  Every wait has a limit (zr_tc.cuh); when one runs out the CTA's
// remaining rows become NaN.
#include "zr_attn_tc.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

constexpr int kFwdThreads = 384;
constexpr uint32_t kFwdRows = 256;

template <int DP>
struct FwdCfg {
  static constexpr uint32_t kTile = DP / 64 * kAtBlock;  // bytes of 128 rows
  static constexpr int kStages = DP == 64 ? 4 : 2;       // of keys, and of values
  // Room for the queries: heads of 64 have it for the next item's too, which arrive
  // while this one is at work.
  static constexpr int kStay = DP == 64 ? 2 : 1;
  static constexpr uint32_t kSmem = 2 * (kStay + kStages) * kTile + 1024;
  static constexpr uint32_t kO = 256;                    // columns: S0, S1, O0, O1
  static constexpr uint32_t kCols = 512;
};

// One share of a pair of tiles' keys: tile h takes the key tiles [first, end(h)),
// of which the one on the diagonal, 2 * tile + h, is its last.
struct FwdRange {
  uint32_t tiles, h0;        // the tiles [h0, tiles) have something in this share
  uint32_t first, end0, end1;
  __device__ __forceinline__ uint32_t end(uint32_t h) const { return h ? end1 : end0; }
};
template <bool SHARES>
__device__ __forceinline__ FwdRange fwd_range(const AttnPlan& p, const AttnTile& t, uint32_t split) {
  FwdRange r;
  r.tiles = t.tile * kFwdRows + 128 < t.len ? 2 : 1;
  if (!SHARES) {
    r.h0 = r.first = 0;
    r.end0 = 2 * t.tile + 1;
    r.end1 = r.tiles == 2 ? r.end0 + 1 : 0;
    return r;
  }
  const uint32_t n = 2 * t.tile + r.tiles;
  r.first = uint32_t(uint64_t(n) * split / p.splits);
  const uint32_t end = uint32_t(uint64_t(n) * (split + 1) / p.splits);
  r.end0 = end < 2 * t.tile + 1 ? end : 2 * t.tile + 1;
  r.end1 = r.tiles == 2 ? end : 0;
  r.h0 = r.end0 > r.first ? 0 : r.end1 > r.first ? 1 : 2;
  return r;
}

// Items: pairs of query tiles (as slots) times heads, or with p.splits shares of
// their keys (SHARES), whose results k_attn_fwd_join weighs.
template <int DP, bool SHARES>
__global__ void __launch_bounds__(kFwdThreads, 1)
    k_attn_fwd(const __grid_constant__ AttnPlan p, const __grid_constant__ AttnMaps maps) {
  using Cfg = FwdCfg<DP>;
  constexpr int S = Cfg::kStages;
  constexpr uint32_t kTile = Cfg::kTile;
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_qfull[2 * Cfg::kStay], s_qempty[2 * Cfg::kStay], s_kfull[S], s_kempty[S], s_vfull[S], s_vempty[S], s_landed;
  __shared__ uint64_t s_sfull[2], s_pfull[2], s_ofull[2], s_oempty[2];
  __shared__ uint32_t s_tmem, s_abort;
  pdl_trigger();
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + 2 * Cfg::kStay * kTile, sv = sk + S * kTile;
  volatile uint32_t* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * Cfg::kStay; ++i) {
      mbar_init(smem_u32(&s_qfull[i]), 1);
      mbar_init(smem_u32(&s_qempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_sfull[i]), 1);
      mbar_init(smem_u32(&s_pfull[i]), 4);
      mbar_init(smem_u32(&s_ofull[i]), 1);
      mbar_init(smem_u32(&s_oempty[i]), 4);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s_kfull[i]), 1);
      mbar_init(smem_u32(&s_kempty[i]), 1);
      mbar_init(smem_u32(&s_vfull[i]), 1);
      mbar_init(smem_u32(&s_vempty[i]), 1);
    }
    mbar_init(smem_u32(&s_landed), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(&s_tmem), Cfg::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  const uint32_t items = p.slots * (SHARES ? p.splits : 1) * p.heads;
  pdl_wait();

  if (warp >= 8) {
    regs_give<72>();
    const bool leader = elect_one();
    bool ok = true;
    if (warp == 8) {
      uint32_t nk = 0, nq[2] = {0, 0}, landed = 0;
      for (uint32_t round = 0; ok && round * gridDim.x < items; ++round) {
        const uint32_t w = at_item(round);
        if (w >= items) continue;
        const uint32_t share = w / p.heads, head = w - share * p.heads, kvh = head / p.group, slot = SHARES ? share / p.splits : share;
        const AttnTile t = attn_tile(p, slot, false);
        if (!t.live) continue;
        const FwdRange run = fwd_range<SHARES>(p, t, share - slot * p.splits);
        if (run.h0 >= run.tiles) continue;
        const uint32_t row0 = t.tile * kFwdRows, end = run.end(run.tiles - 1);
        for (uint32_t i = run.first; i < end && ok; ++i) {
          const uint32_t stage = nk % S, phase = (nk / S) & 1;
          ++nk;
          // Queries with the first keys: each tile's when the last item's scores are done.
          if (i == run.first) {
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
              if (!ok || h < run.h0 || h >= run.tiles) continue;
              const uint32_t room = h + nq[h] % Cfg::kStay * 2;
              ok = warp_wait(smem_u32(&s_qempty[room]), ((nq[h] / Cfg::kStay) & 1) ^ 1, abort);
              ++nq[h];
              if (ok && leader) {
                const uint32_t bar = smem_u32(&s_qfull[room]);
                mbar_expect(bar, kTile);
                for (uint32_t b = 0; b < DP / 64; ++b)
                  at_load(sq + room * kTile + b * kAtBlock, &maps.q, bar, b, head, t.start + row0 + h * 128, t.batch);
              }
              __syncwarp();
            }
          }
          ok = ok && warp_wait(smem_u32(&s_kempty[stage]), phase ^ 1, abort);
          if (!ok) break;
          if (leader) {
            const uint32_t bar = smem_u32(&s_kfull[stage]);
            mbar_expect(bar, kTile);
            for (uint32_t b = 0; b < DP / 64; ++b)
              at_load(sk + stage * kTile + b * kAtBlock, &maps.k, bar, b, kvh, t.start + i * 128, t.batch);
          }
          __syncwarp();
          ok = warp_wait(smem_u32(&s_vempty[stage]), phase ^ 1, abort);
          if (!ok) break;
          const uint32_t full = smem_u32(&s_vfull[stage]);
          const bool cut = p.offsets && (i + 1) * 128 > t.len;  // others' rows behind the sequence
          const uint32_t bar = cut ? smem_u32(&s_landed) : full;
          if (leader) {
            mbar_expect(bar, kTile);
            for (uint32_t b = 0; b < DP / 64; ++b)
              at_load(sv + stage * kTile + b * kAtBlock, &maps.v, bar, b, kvh, t.start + i * 128, t.batch);
          }
          __syncwarp();
          if (cut) {
            ok = warp_wait(bar, landed & 1, abort);
            ++landed;
            if (ok) {
              at_clear(sv + stage * kTile, DP / 64, t.len - i * 128);
              if (leader) mbar_arrive(full);
            }
            __syncwarp();
          }
        }
      }
    } else if (warp == 9) {
      uint32_t n_key = 0, items_of[2] = {0, 0}, tiles_of[2] = {0, 0};
      for (uint32_t round = 0; ok && round * gridDim.x < items; ++round) {
        const uint32_t w = at_item(round);
        if (w >= items) continue;
        const uint32_t share = w / p.heads, slot = SHARES ? share / p.splits : share;
        const AttnTile t = attn_tile(p, slot, false);
        if (!t.live) continue;
        const FwdRange run = fwd_range<SHARES>(p, t, share - slot * p.splits);
        if (run.h0 >= run.tiles) continue;
        // Scores of tile h with key tile i, whose stage goes back with the last tile that reads it.
        auto scores = [&](uint32_t h, uint32_t i) {
          const uint32_t at = n_key + i - run.first, stage = at % S, room = h + items_of[h] % Cfg::kStay * 2;
          ok = ok && warp_wait(smem_u32(&s_kfull[stage]), (at / S) & 1, abort);
          if (i == run.first) ok = ok && warp_wait(smem_u32(&s_qfull[room]), (items_of[h] / Cfg::kStay) & 1, abort);
          if (!ok) return;
          tc_fence_after();
          if (leader) {
            at_scores<DP>(tmem + h * 128, sq + room * kTile, sk + stage * kTile);
            tc_commit<1>(smem_u32(&s_sfull[h]));
            if (i + 1 == run.end(h)) tc_commit<1>(smem_u32(&s_qempty[room]));
            if (h + 1 == run.tiles) tc_commit<1>(smem_u32(&s_kempty[stage]));
          }
          __syncwarp();
        };
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
          if (h >= run.h0 && h < run.tiles) scores(h, run.first);
        const uint32_t end = run.end(run.tiles - 1);
        for (uint32_t i = run.first; i < end && ok; ++i) {
          const uint32_t at = n_key + i - run.first, stage = at % S;
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            if (!ok || h < run.h0 || h >= run.tiles || i >= run.end(h)) continue;
            if (i == run.first) ok = warp_wait(smem_u32(&s_oempty[h]), (items_of[h] & 1) ^ 1, abort);
            ok = ok && warp_wait(smem_u32(&s_vfull[stage]), (at / S) & 1, abort);
            ok = ok && warp_wait(smem_u32(&s_pfull[h]), tiles_of[h] & 1, abort);
            if (!ok) continue;
            ++tiles_of[h];
            tc_fence_after();
            if (leader) {
              at_sum<DP>(tmem + Cfg::kO + h * DP, tmem + h * 128, sv + stage * kTile, i != run.first);
              if (i + 1 == run.end(h)) tc_commit<1>(smem_u32(&s_ofull[h]));
              if (h + 1 == run.tiles) tc_commit<1>(smem_u32(&s_vempty[stage]));
            }
            __syncwarp();
            if (i + 1 < run.end(h)) scores(h, i + 1);
          }
        }
        n_key += end - run.first;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
          if (h >= run.h0 && h < run.tiles) ++items_of[h];
      }
    }
  } else {
    regs_take<216>();
    const uint32_t h = warp >> 2, quad = warp & 3, mine = quad * 32 + lane;
    const uint32_t s_at = tmem + (quad << 21) + h * 128, o_at = tmem + (quad << 21) + Cfg::kO + h * DP;
    const F2 c2 = f2_splat(p.scale_log2);
    bool ok = true;
    uint32_t n_item = 0, n_tile = 0;
    for (uint32_t round = 0; round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t share = w / p.heads, head = w - share * p.heads, slot = SHARES ? share / p.splits : share;
      const AttnTile t = attn_tile(p, slot, false);
      if (!t.live) continue;
      const uint32_t split = SHARES ? share - slot * p.splits : 0;
      const FwdRange run = fwd_range<SHARES>(p, t, split);
      if (h < run.h0 || h >= run.tiles) continue;  // k_attn_fwd_join knows
      const uint32_t row = t.tile * kFwdRows + h * 128 + mine, last = 2 * t.tile + h;
      float top = -INFINITY, off = 0.f;  // the row's maximum so far; -top * scale * log2(e)
      float sum = 0.f;
      for (uint32_t i = run.first; i < run.end(h); ++i, ++n_tile) {
        ok = ok && warp_wait(smem_u32(&s_sfull[h]), n_tile & 1, abort);
        if (!ok) break;
        tc_fence_after();
        float v[128];
        {
          uint32_t r[128];
#pragma unroll
          for (int j = 0; j < 4; ++j) tc_load32_async(s_at + j * 32, r + j * 32);
          tc_wait_load();
#pragma unroll
          for (int j = 0; j < 128; ++j) v[j] = __uint_as_float(r[j]);
        }
        if (i == last) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (uint32_t(j) > mine) v[j] = -INFINITY;
        }
        float m[4] = {top, v[0], v[1], v[2]};
#pragma unroll
        for (int j = 3; j < 127; j += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            m[k] = j + 4 + k < 128 ? fmaxf(fmaxf(m[k], v[j + k]), v[j + 4 + k]) : fmaxf(m[k], v[j + k]);
        }
        m[0] = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), v[127]);
        const float off_new = m[0] == -INFINITY ? 0.f : -(m[0] * p.scale_log2);
        if (i > run.first && __any_sync(0xFFFFFFFFu, m[0] > top)) {
          const float keep = m[0] > top ? ex2(__fmaf_rn(top, p.scale_log2, off_new)) : 1.f;
          sum *= keep;
          const F2 f = f2_splat(keep);
#pragma unroll
          for (int j = 0; j < DP; j += 32) {
            uint32_t r[32];
            tc_load32_async(o_at + j, r);
            tc_wait_load();
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float lo, hi;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), f), lo, hi);
              r[k] = __float_as_uint(lo);
              r[k + 1] = __float_as_uint(hi);
            }
            tc_store32(o_at + j, r);
          }
        }
        top = m[0];
        off = off_new;
        const F2 off2 = f2_splat(off);
        F2 add[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) add[k] = f2_splat(0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t r[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float lo, hi;
            f2_unpack(f2_fma(f2_pack(v[j * 64 + 2 * k], v[j * 64 + 2 * k + 1]), c2, off2), lo, hi);
            lo = ex2(lo);
            hi = ex2(hi);
            add[k & 3] = f2_add(add[k & 3], f2_pack(lo, hi));
            r[k] = pack_bf16(lo, hi);
          }
          tc_store32(s_at + j * 32, r);
        }
        tc_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_pfull[h]));
        float lo, hi;
        f2_unpack(f2_add(f2_add(add[0], add[1]), f2_add(add[2], add[3])), lo, hi);
        sum += lo + hi;
      }
      ok = ok && warp_wait(smem_u32(&s_ofull[h]), n_item & 1, abort);
      ++n_item;
      tc_fence_after();
      const float by = ok ? 1.f / sum : qnan();
      const int64_t token = int64_t(t.start) + row;
      const int64_t flat = (int64_t(t.batch) * p.tokens + token) * p.heads + head;
      const float lse = ok ? (log2f(sum) - off) * 0.6931471805599453f : qnan();
      const int64_t rows = int64_t(p.batch) * p.tokens * p.heads;
      float* part = p.part + (split * rows + flat) * DP;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(const_cast<void*>(p.o.p)) + int64_t(t.batch) * p.o.batch +
                         token * p.o.token + int64_t(head) * p.o.head;
      __nv_bfloat16* low = p.low ? static_cast<__nv_bfloat16*>(p.low) + flat * p.dim : nullptr;
#pragma unroll
      for (int j = 0; j < DP; j += 32) {
        float x[32];
        __syncwarp();
        tc_load32(o_at + j, x);
        if (j + 32 >= DP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_oempty[h]));
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] *= by;
        if (SHARES) {
          if (row < t.len) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(part + j + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          }
        } else if (row < t.len) {
          at_store_row(o, p.o.elem, p.o_wide, x, j, p.dim);
          if (low) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] -= __bfloat162float(__float2bfloat16_rn(x[k]));
            at_store_row(low, 1, p.low_wide, x, j, p.dim);
          }
        }
      }
      if (row < t.len) {
        if (SHARES) p.part[p.splits * rows * DP + split * rows + flat] = lse;
        else if (p.lse) p.lse[flat] = lse;
      }
    }
  }
  __syncthreads();
  if (*abort) {
    // Copies and products still in flight land within this time.
    const uint64_t t0 = timer_ns();
    while (timer_ns() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free<1>(tmem, Cfg::kCols);
}

// Weighs the shares' results by their sums: four elements a thread, blockIdx.x =
// (slot * heads + head) * (blocks of a pair of tiles) + block.
template <int DP>
__global__ void __launch_bounds__(kThreads) k_attn_fwd_join(const __grid_constant__ AttnPlan p) {
  constexpr uint32_t kRows = kThreads / (DP / 4), kBlocks = kFwdRows / kRows;
  pdl_wait();
  const uint32_t item = blockIdx.x / kBlocks, slot = item / p.heads, head = item - slot * p.heads;
  const AttnTile t = attn_tile(p, slot, false);
  const uint32_t in = blockIdx.x % kBlocks * kRows + threadIdx.x / (DP / 4), d = threadIdx.x % (DP / 4) * 4;
  const uint32_t row = t.tile * kFwdRows + in;
  if (!t.live || row >= t.len) return;
  const int64_t rows = int64_t(p.batch) * p.tokens * p.heads;
  const int64_t flat = (int64_t(t.batch) * p.tokens + t.start + row) * p.heads + head;
  float4 x[8];
  float l[8], top = -INFINITY;
#pragma unroll
  for (uint32_t split = 0; split < 8; ++split) {
    l[split] = -INFINITY;
    x[split] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (split >= p.splits) continue;
    const FwdRange run = fwd_range<true>(p, t, split);
    if (in / 128 < run.h0 || in / 128 >= run.tiles) continue;
    l[split] = p.part[p.splits * rows * DP + split * rows + flat];
    x[split] = *reinterpret_cast<const float4*>(p.part + (split * rows + flat) * DP + d);
    top = fmaxf(top, l[split]);
  }
  float sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int split = 0; split < 8; ++split) {
    const float w = l[split] == -INFINITY ? 0.f : ex2_full((l[split] - top) * kLog2e);
    sum += w;
    y[0] = __fmaf_rn(w, x[split].x, y[0]);
    y[1] = __fmaf_rn(w, x[split].y, y[1]);
    y[2] = __fmaf_rn(w, x[split].z, y[2]);
    y[3] = __fmaf_rn(w, x[split].w, y[3]);
  }
  const float by = 1.f / sum;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(const_cast<void*>(p.o.p)) + int64_t(t.batch) * p.o.batch +
                     (int64_t(t.start) + row) * p.o.token + int64_t(head) * p.o.head;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (d + k >= p.dim) continue;
    const float v = y[k] * by;
    const __nv_bfloat16 r = __float2bfloat16_rn(v);
    o[int64_t(d + k) * p.o.elem] = r;
    if (p.low) static_cast<__nv_bfloat16*>(p.low)[flat * p.dim + d + k] = __float2bfloat16_rn(v - __bfloat162float(r));
  }
  if (p.lse && d == 0) p.lse[flat] = top + logf(sum);
}

template <int DP>
cudaError_t launch(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  constexpr size_t smem = FwdCfg<DP>::kSmem;
  const auto k = p.splits > 1 ? k_attn_fwd<DP, true> : k_attn_fwd<DP, false>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  const uint32_t items = p.slots * p.splits * p.heads;
  e = launch_k(k, items < kSms ? items : kSms, kFwdThreads, smem, s, p, maps);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_k(k_attn_fwd_join<DP>, p.slots * p.heads * (DP / 4), kThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  return p.dim <= 64 ? launch<64>(p, maps, s) : launch<128>(p, maps, s);
}

}  // namespace zr
