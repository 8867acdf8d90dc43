// zr_attn_bwd.cu — causal attention, backward, on the tensor cores.
//
// Two kernels, each of which computes the scores again and keeps its results in
// tensor memory to the end: a tile of 128 keys with all queries that see it for
// grad_k and grad_v (k_attn_kv), a tile of 128 queries with all its keys for
// grad_q (k_attn_q).  Seven products for the five it cannot do without, and in
// return every gradient is one sum in a fixed order: no atomics, no partial sums in
// memory.  In k_attn_kv the scores are taken transposed, keys along the lanes, so
// that weights and their gradients lie in tensor memory as the products need them:
// as A operands, written over the scores they come from.
//
// Warp 8 brings operands by TMA, warp 9 issues, warp 10 brings the rows' lse and
// delta (k_attn_kv), and the warps 0-3 and 4-7 take 64 of a tile's 128 columns each, a lane
// per thread.  With s the scores and d the products grad_out . v of a step:
//   tensor core:  dV(i) += P(i) dO   s(i+1) | dK(i) += dS(i) Q   d(i+1)
//   warps:        dS(i) from d(i), P(i)     | P(i+1) from s(i+1)
// so that both work at all times ([2, 8192] tokens of 16 heads of 128, 1470 us: the
// products that are computed at 1.3 PFLOP/s; four groups of 32 columns instead
// of two of 64, for more warps, took 1 to 3 % longer); in k_attn_q likewise, with s(i+1) as soon as
// s(i) has been read.  Every wait has a limit (zr_tc.cuh); when one runs out the
// CTA's remaining rows become NaN.
#include "zr_attn_tc.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

constexpr int kBwdThreads = 384;

template <int DP>
struct BwdCfg {
  static constexpr uint32_t kTile = DP / 64 * kAtBlock;
  static constexpr int kStages = DP == 64 ? 3 : 2;  // of two tiles
  // Room for the tiles that stay: heads of 64 have it for the next item's too, which
  // arrive while this one is at work.
  static constexpr int kStay = DP == 64 ? 2 : 1;
  static constexpr uint32_t kSmem = 2 * (kStay + kStages) * kTile + 1024;
  static constexpr uint32_t kS = 0, kD = 128, kAcc = 256, kCols = 512;
};

// W [128, 128] as bfloat16 in two halves of 32 columns, 64 columns apart.
template <int DP>
__device__ __forceinline__ void bwd_sum(uint32_t d, uint32_t w, uint32_t b, bool accumulate) {
  const uint64_t db = at_desc(b, true);
#pragma unroll
  for (uint32_t j = 0; j < kAtRows / 16; ++j)
    tc_mma_ts(d, w + (j / 4) * 64 + (j % 4) * 8, db + j * (2048 >> 4), at_idesc(DP, true), accumulate || j != 0);
}

__device__ __forceinline__ void bwd_read64(uint32_t addr, float* v) {
  uint32_t r[64];
  tc_load32_async(addr, r);
  tc_load32_async(addr + 32, r + 32);
  tc_wait_load();
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void bwd_write64(uint32_t addr, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  tc_store32(addr, r);
  tc_wait_store();
}
// By a whole warp: what it read and wrote in tensor memory is done.
__device__ __forceinline__ void bwd_arrive(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// The rows of a gradient out of tensor memory, times `by`.
template <int DP>
__device__ __forceinline__ void bwd_store(const AttnPlan& p, const AttnView& x, uint32_t addr, const AttnTile& t, uint32_t row,
                                          uint32_t head, float by, bool is_wide) {
  const bool live = row < t.len && x.p != nullptr;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(const_cast<void*>(x.p)) + int64_t(t.batch) * x.batch +
                     (int64_t(t.start) + row) * x.token + int64_t(head) * x.head;
#pragma unroll
  for (int j = 0; j < DP; j += 32) {
    float v[32];
    __syncwarp();
    tc_load32(addr + j, v);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] *= by;
    if (live) at_store_row(o, x.elem, is_wide, v, j, p.dim);
  }
}

// The steps of one share of a key tile: queries' tiles of the group's heads, counted through.
struct KvSteps {
  uint32_t per, first, count;  // steps of a head; the share's first, how many
};
__device__ __forceinline__ KvSteps kv_steps(const AttnPlan& p, const AttnTile& t, uint32_t split) {
  const uint32_t per = (t.len + 127) / 128 - t.tile, all = per * p.group;
  const uint32_t first = uint32_t(uint64_t(all) * split / p.splits);
  return {per, first, uint32_t(uint64_t(all) * (split + 1) / p.splits) - first};
}
// A row's sums of one share in the workspace: grad_v, then grad_k, DP each.
template <int DP>
__device__ __forceinline__ float* part_row(const AttnPlan& p, uint32_t split, const AttnTile& t, uint32_t row, uint32_t kvh) {
  const int64_t at = (int64_t(t.batch) * p.tokens + t.start + row) * p.kv_heads + kvh;
  return p.part + (int64_t(split) * p.batch * p.tokens * p.kv_heads + at) * (2 * DP);
}

// Items: key tiles (as slots) times kv_heads, or with p.splits shares of their steps,
// whose sums k_attn_join adds.
template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_kv(const __grid_constant__ AttnPlan p, const __grid_constant__ AttnMaps maps) {
  using Cfg = BwdCfg<DP>;
  constexpr int S = Cfg::kStages;
  constexpr uint32_t kTile = Cfg::kTile;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(16) float s_rows[2][256];  // -lse2 and -delta of a tile of queries
  __shared__ uint64_t s_kvfull[Cfg::kStay], s_kvempty[Cfg::kStay], s_full[S], s_empty[S], s_landed, s_rfull[2], s_rempty[2];
  __shared__ uint64_t s_sfull, s_pfull, s_dfull, s_wfull, s_accfull, s_accempty;
  __shared__ uint32_t s_tmem, s_abort;
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t stay = (smem_u32(s_raw) + 1023u) & ~1023u, ring = stay + Cfg::kStay * 2 * kTile;
  volatile uint32_t* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kStay; ++i) {
      mbar_init(smem_u32(&s_kvfull[i]), 1);
      mbar_init(smem_u32(&s_kvempty[i]), 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 1);
    }
    mbar_init(smem_u32(&s_landed), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_rfull[i]), 1);
      mbar_init(smem_u32(&s_rempty[i]), 8);
    }
    mbar_init(smem_u32(&s_sfull), 1);
    mbar_init(smem_u32(&s_pfull), 8);
    mbar_init(smem_u32(&s_dfull), 1);
    mbar_init(smem_u32(&s_wfull), 8);
    mbar_init(smem_u32(&s_accfull), 1);
    mbar_init(smem_u32(&s_accempty), 8);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(&s_tmem), Cfg::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  const uint32_t items = p.slots * p.splits * p.kv_heads;
  pdl_wait();
  pdl_trigger();  // behind the wait: k_attn_q may start beside this one, the rows are done

  if (warp >= 8) {
    regs_give<72>();
    const bool leader = elect_one();
    bool ok = true;
    uint32_t n_item = 0, n_step = 0, landed = 0;
    for (uint32_t round = 0; warp < 11 && ok && round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t share = w / p.kv_heads, kvh = w - share * p.kv_heads, slot = share / p.splits;
      const AttnTile t = attn_tile(p, slot, true);
      if (!t.live) continue;
      const uint32_t tiles = (t.len + 127) / 128;
      const KvSteps run = kv_steps(p, t, share - slot * p.splits);
      const uint32_t steps = run.count;
      if (steps == 0) continue;
      const uint32_t sk = stay + n_item % Cfg::kStay * 2 * kTile, sv = sk + kTile;
      if (warp == 8) {
        ok = warp_wait(smem_u32(&s_kvempty[n_item % Cfg::kStay]), ((n_item / Cfg::kStay) & 1) ^ 1, abort);
        if (!ok) break;
        if (leader) {
          const uint32_t bar = smem_u32(&s_kvfull[n_item % Cfg::kStay]);
          mbar_expect(bar, 2 * kTile);
          for (uint32_t b = 0; b < DP / 64; ++b) {
            at_load(sk + b * kAtBlock, &maps.k, bar, b, kvh, t.start + t.tile * 128, t.batch);
            at_load(sv + b * kAtBlock, &maps.v, bar, b, kvh, t.start + t.tile * 128, t.batch);
          }
        }
        __syncwarp();
        uint32_t head = kvh * p.group + run.first / run.per, q = t.tile + run.first % run.per;
        for (uint32_t i = 0; i < steps; ++i, ++n_step) {
          const uint32_t stage = n_step % S, sq = ring + stage * 2 * kTile;
          ok = warp_wait(smem_u32(&s_empty[stage]), ((n_step / S) & 1) ^ 1, abort);
          if (!ok) break;
          const bool cut = p.offsets && (q + 1) * 128 > t.len;  // others' rows behind the sequence
          const uint32_t full = smem_u32(&s_full[stage]), bar = cut ? smem_u32(&s_landed) : full;
          if (leader) {
            mbar_expect(bar, 2 * kTile);
            for (uint32_t b = 0; b < DP / 64; ++b) {
              at_load(sq + b * kAtBlock, &maps.q, bar, b, head, t.start + q * 128, t.batch);
              at_load(sq + kTile + b * kAtBlock, &maps.go, bar, b, head, t.start + q * 128, t.batch);
            }
          }
          __syncwarp();
          if (cut) {
            ok = warp_wait(bar, landed & 1, abort);
            ++landed;
            if (!ok) break;
            at_clear(sq, DP / 64, t.len - q * 128);
            at_clear(sq + kTile, DP / 64, t.len - q * 128);
            if (leader) mbar_arrive(full);
            __syncwarp();
          }
          if (++q == tiles) {
            q = t.tile;
            ++head;
          }
        }
      } else if (warp == 9) {
        ok = warp_wait(smem_u32(&s_kvfull[n_item % Cfg::kStay]), (n_item / Cfg::kStay) & 1, abort);
        auto stage_at = [&](uint32_t i) { return ring + (n_step + i) % S * 2 * kTile; };
        auto scores = [&](uint32_t i) {  // of step i, when its operands are there
          ok = ok && warp_wait(smem_u32(&s_full[(n_step + i) % S]), ((n_step + i) / S) & 1, abort);
          if (!ok) return;
          tc_fence_after();
          if (leader) {
            at_scores<DP>(tmem + Cfg::kS, sk, stage_at(i));
            tc_commit<1>(smem_u32(&s_sfull));
          }
          __syncwarp();
        };
        auto products = [&](uint32_t i) {
          if (leader) {
            at_scores<DP>(tmem + Cfg::kD, sv, stage_at(i) + kTile);
            tc_commit<1>(smem_u32(&s_dfull));
          }
          __syncwarp();
        };
        scores(0);
        if (ok) products(0);
        for (uint32_t i = 0; i < steps && ok; ++i) {
          ok = warp_wait(smem_u32(&s_pfull), (n_step + i) & 1, abort);
          if (ok && i == 0) ok = warp_wait(smem_u32(&s_accempty), (n_item & 1) ^ 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) bwd_sum<DP>(tmem + Cfg::kAcc, tmem + Cfg::kS, stage_at(i) + kTile, i != 0);
          __syncwarp();
          if (i + 1 < steps) scores(i + 1);
          ok = ok && warp_wait(smem_u32(&s_wfull), (n_step + i) & 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            bwd_sum<DP>(tmem + Cfg::kAcc + DP, tmem + Cfg::kD, stage_at(i), i != 0);
            tc_commit<1>(smem_u32(&s_empty[(n_step + i) % S]));
            if (i + 1 == steps) {
              tc_commit<1>(smem_u32(&s_accfull));
              tc_commit<1>(smem_u32(&s_kvempty[n_item % Cfg::kStay]));
            }
          }
          __syncwarp();
          if (i + 1 < steps) products(i + 1);
        }
        n_step += steps;
      } else {
        uint32_t head = kvh * p.group + run.first / run.per, q = t.tile + run.first % run.per;
        for (uint32_t i = 0; i < steps; ++i, ++n_step) {
          const uint32_t stage = n_step & 1;
          ok = warp_wait(smem_u32(&s_rempty[stage]), ((n_step / 2) & 1) ^ 1, abort);
          if (!ok) break;
          const int64_t at = (int64_t(t.batch) * p.heads + head) * p.row_pitch + t.start + q * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t r = lane + 32 * k;
            const bool in = q * 128 + r < t.len;  // behind the end the weight is 0
            s_rows[stage][r] = in ? -__ldcg(p.lse2 + at + r) : -INFINITY;
            s_rows[stage][128 + r] = in ? -__ldcg(p.delta + at + r) : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_rfull[stage]));
          if (++q == tiles) {
            q = t.tile;
            ++head;
          }
        }
      }
      ++n_item;
    }
  } else {
    regs_take<216>();
    const uint32_t half = warp >> 2, quad = warp & 3, mine = quad * 32 + lane;
    const uint32_t lanes = tmem + (quad << 21);
    const F2 c2 = f2_splat(p.scale_log2);
    bool ok = true;
    uint32_t n_item = 0, n_step = 0;
    for (uint32_t round = 0; round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t share = w / p.kv_heads, kvh = w - share * p.kv_heads, slot = share / p.splits;
      const AttnTile t = attn_tile(p, slot, true);
      if (!t.live) continue;
      const uint32_t split = share - slot * p.splits;
      const KvSteps run = kv_steps(p, t, split);
      const uint32_t per = run.per, steps = run.count;
      if (steps == 0) continue;  // k_attn_join knows
      uint32_t q = run.first % per;
      for (uint32_t i = 0; i < steps; ++i, ++n_step) {
        const uint32_t stage = n_step & 1;
        const float* rows = s_rows[stage] + half * 64;
        ok = ok && warp_wait(smem_u32(&s_rfull[stage]), (n_step / 2) & 1, abort);
        ok = ok && warp_wait(smem_u32(&s_sfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
        float v[64], d[64];
        bwd_read64(lanes + Cfg::kS + half * 64, v);
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(rows + j);
          f2_unpack(f2_fma(f2_pack(v[j], v[j + 1]), c2, f2_pack(l.x, l.y)), v[j], v[j + 1]);
          f2_unpack(f2_fma(f2_pack(v[j + 2], v[j + 3]), c2, f2_pack(l.z, l.w)), v[j + 2], v[j + 3]);
        }
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = ex2(v[j]);
        if (q == 0) {  // the tile on the diagonal
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (half * 64 + j < mine) v[j] = 0.f;
        }
        bwd_write64(lanes + Cfg::kS + half * 64, v);
        bwd_arrive(smem_u32(&s_pfull));
        ok = warp_wait(smem_u32(&s_dfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
        bwd_read64(lanes + Cfg::kD + half * 64, d);
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(rows + 128 + j);
          f2_unpack(f2_mul(f2_add(f2_pack(d[j], d[j + 1]), f2_pack(l.x, l.y)), f2_pack(v[j], v[j + 1])), d[j], d[j + 1]);
          f2_unpack(f2_mul(f2_add(f2_pack(d[j + 2], d[j + 3]), f2_pack(l.z, l.w)), f2_pack(v[j + 2], v[j + 3])), d[j + 2],
                    d[j + 3]);
        }
        bwd_write64(lanes + Cfg::kD + half * 64, d);
        bwd_arrive(smem_u32(&s_wfull));
        if (lane == 0) mbar_arrive(smem_u32(&s_rempty[stage]));
        if (++q == per) q = 0;
      }
      ok = ok && warp_wait(smem_u32(&s_accfull), n_item & 1, abort);
      ++n_item;
      tc_fence_after();
      const uint32_t row = t.tile * 128 + mine;
      if (p.splits > 1) {
        float* to = part_row<DP>(p, split, t, row, kvh) + half * DP;
#pragma unroll
        for (int j = 0; j < DP; j += 32) {
          float x[32];
          __syncwarp();
          tc_load32(lanes + Cfg::kAcc + half * DP + j, x);
          if (row < t.len) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(to + j + k) =
                  ok ? make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]) : make_float4(qnan(), qnan(), qnan(), qnan());
          }
        }
      } else if (half == 0) {
        bwd_store<DP>(p, p.gv, lanes + Cfg::kAcc, t, row, kvh, ok ? 1.f : qnan(), p.g_wide & 4);
      } else {
        bwd_store<DP>(p, p.gk, lanes + Cfg::kAcc + DP, t, row, kvh, ok ? p.scale : qnan(), p.g_wide & 2);
      }
      bwd_arrive(smem_u32(&s_accempty));
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

// Adds the shares' sums in their order: blockIdx.x = (slot * kv_heads + kv head) *
// 16 + eighth rows, four elements a thread.
template <int DP>
__global__ void __launch_bounds__(kThreads) k_attn_join(const __grid_constant__ AttnPlan p) {
  pdl_wait();
  const uint32_t tile = blockIdx.x / 16, slot = tile / p.kv_heads, kvh = tile - slot * p.kv_heads;
  const AttnTile t = attn_tile(p, slot, true);
  if (!t.live) return;
  for (uint32_t i = threadIdx.x; i < 8 * 2 * DP / 4; i += kThreads) {
    const uint32_t e = i % (2 * DP / 4) * 4, d = e % DP, row = t.tile * 128 + blockIdx.x % 16 * 8 + i / (2 * DP / 4);
    if (row >= t.len || d >= p.dim) continue;
    float4 x[8];
#pragma unroll
    for (uint32_t split = 0; split < 8; ++split)
      x[split] = split < p.splits && kv_steps(p, t, split).count
                     ? *reinterpret_cast<const float4*>(part_row<DP>(p, split, t, row, kvh) + e)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int split = 0; split < 8; ++split) {
      sum[0] += x[split].x; sum[1] += x[split].y; sum[2] += x[split].z; sum[3] += x[split].w;
    }
    const AttnView& g = e < DP ? p.gv : p.gk;
    if (!g.p) continue;
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(const_cast<void*>(g.p)) + int64_t(t.batch) * g.batch +
                        (int64_t(t.start) + row) * g.token + int64_t(kvh) * g.head + int64_t(d) * g.elem;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (d + k < p.dim) to[k * g.elem] = __float2bfloat16_rn(e < DP ? sum[k] : sum[k] * p.scale);
  }
}

// Items: query tiles (as slots) times heads.
template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_q(const __grid_constant__ AttnPlan p, const __grid_constant__ AttnMaps maps) {
  using Cfg = BwdCfg<DP>;
  constexpr int S = Cfg::kStages;
  constexpr uint32_t kTile = Cfg::kTile;
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_qfull[Cfg::kStay], s_qempty[Cfg::kStay], s_full[S], s_empty[S], s_landed;
  __shared__ uint64_t s_sfull, s_sread, s_dfull, s_wfull, s_accfull, s_accempty;
  __shared__ uint32_t s_tmem, s_abort;
  pdl_trigger();
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t stay = (smem_u32(s_raw) + 1023u) & ~1023u, ring = stay + Cfg::kStay * 2 * kTile;
  volatile uint32_t* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kStay; ++i) {
      mbar_init(smem_u32(&s_qfull[i]), 1);
      mbar_init(smem_u32(&s_qempty[i]), 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 1);
    }
    mbar_init(smem_u32(&s_landed), 1);
    mbar_init(smem_u32(&s_sfull), 1);
    mbar_init(smem_u32(&s_sread), 8);
    mbar_init(smem_u32(&s_dfull), 1);
    mbar_init(smem_u32(&s_wfull), 8);
    mbar_init(smem_u32(&s_accfull), 1);
    mbar_init(smem_u32(&s_accempty), 8);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(&s_tmem), Cfg::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  const uint32_t items = p.slots * p.heads;
  // Behind k_attn_kv, of which nothing here depends, this kernel takes the SMs that
  // one leaves: by then the rows' kernel, whose results both read, is done (k_attn_kv
  // has waited for it).  It waits at its end instead, so that whatever comes
  // next finds both done.
  const bool beside = (p.want & 6) && p.splits == 1;
  if (!beside) pdl_wait();

  if (warp >= 8) {
    regs_give<72>();
    const bool leader = elect_one();
    bool ok = true;
    uint32_t n_item = 0, n_step = 0, landed = 0;
    for (uint32_t round = 0; warp < 10 && ok && round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t slot = w / p.heads, head = w - slot * p.heads, kvh = head / p.group;
      const AttnTile t = attn_tile(p, slot, false);
      if (!t.live) continue;
      const uint32_t steps = t.tile + 1;
      const uint32_t sq = stay + n_item % Cfg::kStay * 2 * kTile, sg = sq + kTile;
      if (warp == 8) {
        ok = warp_wait(smem_u32(&s_qempty[n_item % Cfg::kStay]), ((n_item / Cfg::kStay) & 1) ^ 1, abort);
        if (!ok) break;
        if (leader) {
          const uint32_t bar = smem_u32(&s_qfull[n_item % Cfg::kStay]);
          mbar_expect(bar, 2 * kTile);
          for (uint32_t b = 0; b < DP / 64; ++b) {
            at_load(sq + b * kAtBlock, &maps.q, bar, b, head, t.start + t.tile * 128, t.batch);
            at_load(sg + b * kAtBlock, &maps.go, bar, b, head, t.start + t.tile * 128, t.batch);
          }
        }
        __syncwarp();
        for (uint32_t i = 0; i < steps; ++i, ++n_step) {
          const uint32_t stage = n_step % S, sk = ring + stage * 2 * kTile;
          ok = warp_wait(smem_u32(&s_empty[stage]), ((n_step / S) & 1) ^ 1, abort);
          if (!ok) break;
          const bool cut = p.offsets && (i + 1) * 128 > t.len;  // others' rows behind the sequence
          const uint32_t full = smem_u32(&s_full[stage]), bar = cut ? smem_u32(&s_landed) : full;
          if (leader) {
            mbar_expect(bar, 2 * kTile);
            for (uint32_t b = 0; b < DP / 64; ++b) {
              at_load(sk + b * kAtBlock, &maps.k, bar, b, kvh, t.start + i * 128, t.batch);
              at_load(sk + kTile + b * kAtBlock, &maps.v, bar, b, kvh, t.start + i * 128, t.batch);
            }
          }
          __syncwarp();
          if (cut) {
            ok = warp_wait(bar, landed & 1, abort);
            ++landed;
            if (!ok) break;
            at_clear(sk, DP / 64, t.len - i * 128);
            if (leader) mbar_arrive(full);
            __syncwarp();
          }
        }
      } else {
        ok = warp_wait(smem_u32(&s_qfull[n_item % Cfg::kStay]), (n_item / Cfg::kStay) & 1, abort);
        auto stage_at = [&](uint32_t i) { return ring + (n_step + i) % S * 2 * kTile; };
        auto scores = [&](uint32_t i) {  // of step i, when its operands are there
          ok = ok && warp_wait(smem_u32(&s_full[(n_step + i) % S]), ((n_step + i) / S) & 1, abort);
          if (!ok) return;
          tc_fence_after();
          if (leader) {
            at_scores<DP>(tmem + Cfg::kS, sq, stage_at(i));
            tc_commit<1>(smem_u32(&s_sfull));
          }
          __syncwarp();
        };
        auto products = [&](uint32_t i) {
          if (leader) {
            at_scores<DP>(tmem + Cfg::kD, sg, stage_at(i) + kTile);
            tc_commit<1>(smem_u32(&s_dfull));
          }
          __syncwarp();
        };
        scores(0);
        if (ok) products(0);
        for (uint32_t i = 0; i < steps && ok; ++i) {
          ok = warp_wait(smem_u32(&s_sread), (n_step + i) & 1, abort);
          if (ok) tc_fence_after();
          if (i + 1 < steps) scores(i + 1);
          ok = ok && warp_wait(smem_u32(&s_wfull), (n_step + i) & 1, abort);
          if (ok && i == 0) ok = warp_wait(smem_u32(&s_accempty), (n_item & 1) ^ 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            bwd_sum<DP>(tmem + Cfg::kAcc, tmem + Cfg::kD, stage_at(i), i != 0);
            tc_commit<1>(smem_u32(&s_empty[(n_step + i) % S]));
            if (i + 1 == steps) {
              tc_commit<1>(smem_u32(&s_accfull));
              tc_commit<1>(smem_u32(&s_qempty[n_item % Cfg::kStay]));
            }
          }
          __syncwarp();
          if (i + 1 < steps) products(i + 1);
        }
        n_step += steps;
      }
      ++n_item;
    }
  } else {
    regs_take<216>();
    const uint32_t half = warp >> 2, quad = warp & 3, mine = quad * 32 + lane;
    const uint32_t lanes = tmem + (quad << 21);
    const F2 c2 = f2_splat(p.scale_log2);
    bool ok = true;
    uint32_t n_item = 0, n_step = 0;
    for (uint32_t round = 0; round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t slot = w / p.heads, head = w - slot * p.heads;
      const AttnTile t = attn_tile(p, slot, false);
      if (!t.live) continue;
      const uint32_t row = t.tile * 128 + mine;
      const int64_t at = (int64_t(t.batch) * p.heads + head) * p.row_pitch + t.start + row;
      const F2 lse = f2_splat(row < t.len ? -__ldcg(p.lse2 + at) : 0.f),
               delta = f2_splat(row < t.len ? -__ldcg(p.delta + at) : 0.f);
      for (uint32_t i = 0; i <= t.tile; ++i, ++n_step) {
        ok = ok && warp_wait(smem_u32(&s_sfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
        float v[64], d[64];
        bwd_read64(lanes + Cfg::kS + half * 64, v);
        bwd_arrive(smem_u32(&s_sread));
#pragma unroll
        for (int j = 0; j < 64; j += 2) f2_unpack(f2_fma(f2_pack(v[j], v[j + 1]), c2, lse), v[j], v[j + 1]);
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = ex2(v[j]);
        ok = warp_wait(smem_u32(&s_dfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
        bwd_read64(lanes + Cfg::kD + half * 64, d);
#pragma unroll
        for (int j = 0; j < 64; j += 2)
          f2_unpack(f2_mul(f2_add(f2_pack(d[j], d[j + 1]), delta), f2_pack(v[j], v[j + 1])), d[j], d[j + 1]);
        if (i == t.tile) {  // the tile on the diagonal
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (half * 64 + j > mine) d[j] = 0.f;
        }
        bwd_write64(lanes + Cfg::kD + half * 64, d);
        bwd_arrive(smem_u32(&s_wfull));
      }
      ok = ok && warp_wait(smem_u32(&s_accfull), n_item & 1, abort);
      ++n_item;
      tc_fence_after();
      // Each half stores its share of the elements.
      const float by = ok ? p.scale : qnan();
      const bool live = row < t.len;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(const_cast<void*>(p.gq.p)) + int64_t(t.batch) * p.gq.batch +
                         (int64_t(t.start) + row) * p.gq.token + int64_t(head) * p.gq.head;
#pragma unroll
      for (int j = 0; j < DP / 2; j += 32) {
        float x[32];
        const uint32_t e = half * (DP / 2) + j;
        __syncwarp();
        tc_load32(lanes + Cfg::kAcc + e, x);
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] *= by;
        if (live) at_store_row(o, p.gq.elem, p.g_wide & 1, x, e, p.dim);
      }
      bwd_arrive(smem_u32(&s_accempty));
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
  if (beside) pdl_wait();
}

template <typename K>
cudaError_t go(K k, uint32_t items, uint32_t smem, const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), int(smem));
  if (e != cudaSuccess) return e;
  return launch_k(k, items < kSms ? items : kSms, kBwdThreads, smem, s, p, maps);
}

template <int DP>
cudaError_t launch(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.want & 6) e = go(k_attn_kv<DP>, p.slots * p.splits * p.kv_heads, BwdCfg<DP>::kSmem, p, maps, s);
  if (e == cudaSuccess && p.splits > 1) e = launch_k(k_attn_join<DP>, p.slots * p.kv_heads * 16, kThreads, 0, s, p);
  if (e == cudaSuccess && (p.want & 1)) e = go(k_attn_q<DP>, p.slots * p.heads, BwdCfg<DP>::kSmem, p, maps, s);
  return e;
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  return p.dim <= 64 ? launch<64>(p, maps, s) : launch<128>(p, maps, s);
}

}  // namespace zr
