// zr_attn_f32.cu — causal attention of binary32 heads of up to 64 elements on the
// tensor cores, forward and backward.
//
// Each operand is the sum of three bfloat16 parts that hold it to 2^-24, and a
// product the sum of the six products of parts that reach 2^-24 of it, smallest
// first: each is exact in binary32 before the accumulation.  k_attn_split brings q, k, v
// (and grad_out) into parts, [part][batch][token][head][64], where a tile of 128
// rows is one TMA box; the weights and their gradients are split as they are
// written to tensor memory.  The rest is the bfloat16 kernels' (zr_attn_fwd.cu,
// zr_attn_bwd.cu) with two differences.  The tensor core's accumulation truncates, by
// about 1.3 * 2^-24 of the sum per 16 terms, so a tile's result is read and added in
// registers, rounding to nearest, and no sum on the tensor core is longer than
// 128 terms.  And a tile's parts take 48 KB, so there is one stage: what the
// next step reads arrives when this step's products are done.
//
// Bound by the tensor core (six products) and, with that single stage, by a
// load and a round through the weights per step: [2, 2048] tokens of 16 heads of
// 64, 118 us forward and 371 backward, where the binary32 multiply-adds of
// zr_attn_any.cu take 488 and 1561; [16, 255] tokens of 6 heads 24 and 57, there 40 and 123.
#include "zr_attn_tc.cuh"
#include "zr_launch.h"

namespace zr {
namespace {

constexpr int kF32Threads = 384;
constexpr uint32_t kParts = 3;
constexpr uint32_t kTile = kParts * kAtBlock;    // 128 rows of 64 elements
constexpr uint32_t kF32Smem = 4 * kTile + 1024;  // two tiles that stay, two that go past

// The parts (a, b) of the six products in the order they are added.
__device__ __forceinline__ constexpr uint32_t pair_of(int i, int operand) {
  constexpr uint32_t pairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
  return pairs[i][operand];
}
// All parts of 128 tokens of a head.
__device__ __forceinline__ void load_parts(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t head, uint32_t token,
                                           uint32_t batch) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(0), "r"(head), "r"(token), "r"(batch), "r"(0)
      : "memory");
}
// D[128, 128] = A B^T.
__device__ __forceinline__ void scores_of(uint32_t d, uint32_t a, uint32_t b) {
  const uint64_t da = at_desc(a, false), db = at_desc(b, false);
#pragma unroll
  for (int i = 0; i < 6; ++i)
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      tc_mma<1>(d, da + pair_of(i, 0) * (kAtBlock >> 4) + j * 2, db + pair_of(i, 1) * (kAtBlock >> 4) + j * 2,
                at_idesc(128, false), (i | j) != 0);
}
// Where a part of 32 columns' weights goes: over the scores they come from, the
// third part to `more`.
__device__ __forceinline__ uint32_t weights_at(uint32_t s, uint32_t more, uint32_t part, uint32_t chunk) {
  return part < 2 ? s + chunk * 32 + part * 16 : more + chunk * 16;
}
// D[128, 64] = W B, W [128, 128] in parts.
__device__ __forceinline__ void sum_of(uint32_t d, uint32_t s, uint32_t more, uint32_t b) {
  const uint64_t db = at_desc(b, true);
#pragma unroll
  for (int i = 0; i < 6; ++i)
#pragma unroll
    for (uint32_t j = 0; j < kAtRows / 16; ++j)
      tc_mma_ts(d, weights_at(s, more, pair_of(i, 0), j / 2) + (j % 2) * 8,
                db + pair_of(i, 1) * (kAtBlock >> 4) + j * (2048 >> 4), at_idesc(64, true), (i | j) != 0);
}
__device__ __forceinline__ void tc_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 columns' weights in parts; tc_wait_store() before others read.
__device__ __forceinline__ void write_parts(uint32_t s, uint32_t more, uint32_t chunk, const float* x) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = x[i];
#pragma unroll
  for (uint32_t part = 0; part < kParts; ++part) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      if (part < 2) {
        v[2 * i] -= __uint_as_float(r[i] << 16);
        v[2 * i + 1] -= __uint_as_float(r[i] & 0xFFFF0000u);
      }
    }
    tc_store16(weights_at(s, more, part, chunk), r);
  }
}
__device__ __forceinline__ void read32(uint32_t addr, float* v) { tc_load32(addr, v); }
// acc += 32 columns.
__device__ __forceinline__ void add32(uint32_t addr, float* acc) {
  float v[32];
  tc_load32(addr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] += v[i];
}
__device__ __forceinline__ void arrive_warp(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void store_row_f32(float* row, int64_t elem, bool wide, const float* v, uint32_t d0, uint32_t dim) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      if (d0 + i < dim) *reinterpret_cast<float4*>(row + d0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (d0 + i < dim) row[int64_t(d0 + i) * elem] = v[i];
  }
}
__device__ __forceinline__ float* row_of(const AttnView& x, const AttnTile& t, uint32_t row, uint32_t head) {
  return static_cast<float*>(const_cast<void*>(x.p)) + int64_t(t.batch) * x.batch + (int64_t(t.start) + row) * x.token +
         int64_t(head) * x.head;
}
__device__ __forceinline__ void wait_in_flight(volatile uint32_t* abort) {
  if (*abort) {  // copies and products still in flight land within this time
    const uint64_t t0 = timer_ns();
    while (timer_ns() - t0 < 2000000ull) {
    }
  }
}

// ------------------------------------------------------------------ splitting

struct SplitPlan {
  AttnView x[4];             // q, k, v, grad_out
  uint16_t* out[4];          // [part][batch][token][head][W]
  uint32_t heads[4];
  uint64_t first[5];         // first row (batch, token, head) of each, counted through
  uint32_t count, tokens, dim, wide;
  uint32_t beside;           // behind k_attn_rows, on which it does not depend: waits at its end
};

__device__ __forceinline__ float split_load(const float* p) { return *p; }
__device__ __forceinline__ float split_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Rows of W elements, zero behind the head's, eight elements a thread.  PARTS = 1:
// bfloat16 rows that no tensor map describes, as they are.
template <typename E, uint32_t PARTS, uint32_t W>
__global__ void __launch_bounds__(kThreads) k_attn_split(const __grid_constant__ SplitPlan p) {
  constexpr uint32_t kLanes = W / 8;
  pdl_trigger();
  if (!p.beside) pdl_wait();
  const uint64_t i = uint64_t(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (i >= p.first[p.count]) {
    if (p.beside) pdl_wait();
    return;
  }
  uint32_t which = 0;
  while (which + 1 < p.count && i >= p.first[which + 1]) ++which;
  const uint32_t row = uint32_t(i - p.first[which]);  // rows are counted in 31 bits
  const uint32_t e0 = threadIdx.x % kLanes * 8;
  const uint32_t token = row / p.heads[which], head = row - token * p.heads[which], b = token / p.tokens;
  const AttnView& x = p.x[which];
  const E* from = static_cast<const E*>(x.p) + int64_t(b) * x.batch + int64_t(token - b * p.tokens) * x.token +
                  int64_t(head) * x.head;
  float v[8];
  if (sizeof(E) == 4 && p.wide >> which & 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e0 + 4 * h < p.dim) w = *reinterpret_cast<const float4*>(from + e0 + 4 * h);
      v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = e0 + k < p.dim ? split_load(from + int64_t(e0 + k) * x.elem) : 0.f;
  }
  const uint64_t plane = (p.first[which + 1] - p.first[which]) * W;
#pragma unroll
  for (uint32_t part = 0; part < PARTS; ++part) {
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
      v[2 * k] -= __uint_as_float(r[k] << 16);
      v[2 * k + 1] -= __uint_as_float(r[k] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4*>(p.out[which] + part * plane + uint64_t(row) * W + e0) = make_uint4(r[0], r[1], r[2], r[3]);
  }
  if (p.beside) pdl_wait();  // what comes next finds both done
}

// ------------------------------------------------------------------ forward

// Items: pairs of query tiles (as slots of 256 rows) times heads.
__global__ void __launch_bounds__(kF32Threads, 1)
    k_attn_f32_fwd(const __grid_constant__ AttnPlan p, const __grid_constant__ AttnMaps maps) {
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_qfull[2], s_qempty[2], s_kfull, s_kempty, s_vfull, s_vempty, s_landed;
  __shared__ uint64_t s_sfull[2], s_pfull[2], s_ofull[2], s_oempty[2];
  __shared__ uint32_t s_tmem, s_abort;
  constexpr uint32_t kO = 256, kMore = 384;  // columns: S0, S1, O0, O1, third parts
  pdl_trigger();
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t sq = (smem_u32(s_raw) + 1023u) & ~1023u, sk = sq + 2 * kTile, sv = sk + kTile;
  volatile uint32_t* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_qfull[i]), 1);
      mbar_init(smem_u32(&s_qempty[i]), 1);
      mbar_init(smem_u32(&s_sfull[i]), 1);
      mbar_init(smem_u32(&s_pfull[i]), 4);
      mbar_init(smem_u32(&s_ofull[i]), 1);
      mbar_init(smem_u32(&s_oempty[i]), 4);
    }
    for (uint64_t* b : {&s_kfull, &s_kempty, &s_vfull, &s_vempty, &s_landed}) mbar_init(smem_u32(b), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  const uint32_t items = p.slots * p.heads;
  pdl_wait();

  if (warp >= 8) {
    regs_give<104>();
    const bool leader = elect_one();
    bool ok = true;
    if (warp == 8) {
      uint32_t nk = 0, nq[2] = {0, 0}, landed = 0;
      for (uint32_t round = 0; ok && round * gridDim.x < items; ++round) {
        const uint32_t w = at_item(round);
        if (w >= items) continue;
        const uint32_t slot = w / p.heads, head = w - slot * p.heads, kvh = head / p.group;
        const AttnTile t = attn_tile(p, slot, false);
        if (!t.live) continue;
        const uint32_t row0 = t.tile * 256, tiles = row0 + 128 < t.len ? 2 : 1, n = 2 * t.tile + tiles;
        for (uint32_t i = 0; i < n && ok; ++i, ++nk) {
          if (i == 0) {
            for (uint32_t h = 0; h < tiles && ok; ++h) {
              ok = warp_wait(smem_u32(&s_qempty[h]), (nq[h] & 1) ^ 1, abort);
              ++nq[h];
              if (ok && leader) {
                mbar_expect(smem_u32(&s_qfull[h]), kTile);
                load_parts(sq + h * kTile, &maps.q, smem_u32(&s_qfull[h]), head, t.start + row0 + h * 128, t.batch);
              }
              __syncwarp();
            }
          }
          ok = ok && warp_wait(smem_u32(&s_kempty), (nk & 1) ^ 1, abort);
          if (!ok) break;
          if (leader) {
            mbar_expect(smem_u32(&s_kfull), kTile);
            load_parts(sk, &maps.k, smem_u32(&s_kfull), kvh, t.start + i * 128, t.batch);
          }
          __syncwarp();
          ok = warp_wait(smem_u32(&s_vempty), (nk & 1) ^ 1, abort);
          if (!ok) break;
          const bool cut = p.offsets && (i + 1) * 128 > t.len;  // others' rows behind the sequence
          const uint32_t bar = cut ? smem_u32(&s_landed) : smem_u32(&s_vfull);
          if (leader) {
            mbar_expect(bar, kTile);
            load_parts(sv, &maps.v, bar, kvh, t.start + i * 128, t.batch);
          }
          __syncwarp();
          if (cut) {
            ok = warp_wait(bar, landed & 1, abort);
            ++landed;
            if (ok) {
              at_clear(sv, kParts, t.len - i * 128);
              if (leader) mbar_arrive(smem_u32(&s_vfull));
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
        const AttnTile t = attn_tile(p, w / p.heads, false);
        if (!t.live) continue;
        const uint32_t tiles = t.tile * 256 + 128 < t.len ? 2 : 1;
        auto scores = [&](uint32_t h, uint32_t i) {
          ok = ok && warp_wait(smem_u32(&s_kfull), (n_key + i) & 1, abort);
          if (i == 0) ok = ok && warp_wait(smem_u32(&s_qfull[h]), items_of[h] & 1, abort);
          if (!ok) return;
          tc_fence_after();
          if (leader) {
            scores_of(tmem + h * 128, sq + h * kTile, sk);
            tc_commit<1>(smem_u32(&s_sfull[h]));
            if (i == 2 * t.tile + h) tc_commit<1>(smem_u32(&s_qempty[h]));
            if (h + 1 == tiles) tc_commit<1>(smem_u32(&s_kempty));
          }
          __syncwarp();
        };
        for (uint32_t h = 0; h < tiles; ++h) scores(h, 0);
        const uint32_t n = 2 * t.tile + tiles;
        for (uint32_t i = 0; i < n && ok; ++i) {
          for (uint32_t h = 0; h < tiles && ok; ++h) {
            const uint32_t last = 2 * t.tile + h;
            if (i > last) continue;
            if (i == 0) ok = warp_wait(smem_u32(&s_oempty[h]), (items_of[h] & 1) ^ 1, abort);
            ok = ok && warp_wait(smem_u32(&s_vfull), (n_key + i) & 1, abort);
            ok = ok && warp_wait(smem_u32(&s_pfull[h]), tiles_of[h] & 1, abort);
            if (!ok) break;
            ++tiles_of[h];
            tc_fence_after();
            if (leader) {
              sum_of(tmem + kO + h * 64, tmem + h * 128, tmem + kMore + h * 64, sv);
              if (i == last) tc_commit<1>(smem_u32(&s_ofull[h]));
              if (h + 1 == tiles) tc_commit<1>(smem_u32(&s_vempty));
            }
            __syncwarp();
            if (i < last) scores(h, i + 1);
          }
        }
        n_key += n;
        for (uint32_t h = 0; h < tiles; ++h) ++items_of[h];
      }
    }
  } else {
    regs_take<200>();
    const uint32_t h = warp >> 2, quad = warp & 3, mine = quad * 32 + lane;
    const uint32_t lanes = tmem + (quad << 21), s_at = lanes + h * 128, o_at = lanes + kO + h * 64, more = lanes + kMore + h * 64;
    const F2 c2 = f2_splat(p.scale_log2);
    bool ok = true;
    uint32_t n_item = 0, n_tile = 0;
    for (uint32_t round = 0; round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t slot = w / p.heads, head = w - slot * p.heads;
      const AttnTile t = attn_tile(p, slot, false);
      if (!t.live || t.tile * 256 + h * 128 >= t.len) continue;
      const uint32_t row = t.tile * 256 + h * 128 + mine, last = 2 * t.tile + h;
      float top = -INFINITY, sum = 0.f, acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      for (uint32_t i = 0; i <= last; ++i, ++n_tile) {
        ok = ok && warp_wait(smem_u32(&s_sfull[h]), n_tile & 1, abort);
        if (!ok) break;
        tc_fence_after();
        float m = top;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          read32(s_at + c * 32, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (i != last || uint32_t(c * 32 + j) <= mine) m = fmaxf(m, v[j]);
        }
        const float base = m == -INFINITY ? 0.f : m;
        if (i > 0) {  // the last tile's result, whose products are done: these scores come after them
          add32(o_at, acc);
          add32(o_at + 32, acc + 32);
          if (__any_sync(0xFFFFFFFFu, m > top)) {
            const float keep = m > top ? ex2((top - base) * p.scale_log2) : 1.f;
            sum *= keep;
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] *= keep;
          }
        }
        top = m;
        const F2 off = f2_splat(-base);
        F2 add[2] = {f2_splat(0.f), f2_splat(0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          read32(s_at + c * 32, v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            f2_unpack(f2_mul(f2_add(f2_pack(v[j], v[j + 1]), off), c2), v[j], v[j + 1]);
            v[j] = ex2(v[j]);
            v[j + 1] = ex2(v[j + 1]);
            if (i == last) {
              if (uint32_t(c * 32 + j) > mine) v[j] = 0.f;
              if (uint32_t(c * 32 + j + 1) > mine) v[j + 1] = 0.f;
            }
            add[j / 2 & 1] = f2_add(add[j / 2 & 1], f2_pack(v[j], v[j + 1]));
          }
          write_parts(s_at, more, c, v);
        }
        tc_wait_store();
        arrive_warp(smem_u32(&s_pfull[h]));
        float lo, hi;
        f2_unpack(f2_add(add[0], add[1]), lo, hi);
        sum += lo + hi;
      }
      ok = ok && warp_wait(smem_u32(&s_ofull[h]), n_item & 1, abort);
      ++n_item;
      tc_fence_after();
      __syncwarp();
      add32(o_at, acc);
      add32(o_at + 32, acc + 32);
      arrive_warp(smem_u32(&s_oempty[h]));
      const float by = ok ? 1.f / sum : qnan();
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] *= by;
      if (row < t.len) {
        float* o = row_of(p.o, t, row, head);
        store_row_f32(o, p.o.elem, p.o_wide, acc, 0, p.dim);
        store_row_f32(o, p.o.elem, p.o_wide, acc + 32, 32, p.dim);
        if (p.lse)
          p.lse[(int64_t(t.batch) * p.tokens + t.start + row) * p.heads + head] =
              ok ? __fmaf_rn(top, p.scale, logf(sum)) : qnan();
      }
    }
  }
  __syncthreads();
  wait_in_flight(abort);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free<1>(tmem, 512);
}

// ------------------------------------------------------------------ backward

// KV: items are key tiles (slots of 128 rows) times kv_heads, K and V stay, Q and
// grad_out of all queries that see them go past.  Otherwise items are query tiles
// times heads, Q and grad_out stay, K and V go past.  In both s is A B^T of the first
// tiles, d of the second.
template <bool KV>
__global__ void __launch_bounds__(kF32Threads, 1)
    k_attn_f32_bwd(const __grid_constant__ AttnPlan p, const __grid_constant__ AttnMaps maps) {
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(16) float s_rows[2][256];  // KV: -lse and -delta of a tile of queries
  __shared__ uint64_t s_stayfull, s_stayempty, s_full, s_empty, s_landed, s_rfull[2], s_rempty[2];
  __shared__ uint64_t s_sfull, s_pfull, s_dfull, s_wfull, s_accfull, s_accempty;
  __shared__ uint32_t s_tmem, s_abort;
  // Columns: s, d, the sums of the first and of the second weights, third parts of both.
  constexpr uint32_t kD = 128, kAccP = 256, kAccW = 320, kMoreP = 384, kMoreW = 448;
  if (!KV) pdl_trigger();
  const uint32_t warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t stay = (smem_u32(s_raw) + 1023u) & ~1023u, past = stay + 2 * kTile;
  volatile uint32_t* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&s_stayfull, &s_stayempty, &s_full, &s_empty, &s_landed, &s_rfull[0], &s_rfull[1], &s_sfull, &s_dfull,
                        &s_accfull})
      mbar_init(smem_u32(b), 1);
    for (uint64_t* b : {&s_rempty[0], &s_rempty[1], &s_pfull, &s_wfull, &s_accempty}) mbar_init(smem_u32(b), 8);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  const uint32_t per_slot = KV ? p.kv_heads : p.heads, items = p.slots * per_slot;
  // The kernel for grad_q starts on the SMs that the other one leaves, and waits for
  // it at its end (zr_attn_bwd.cu, k_attn_q).
  const bool beside = !KV && (p.want & 6);
  if (!beside) pdl_wait();
  if (KV) pdl_trigger();

  if (warp >= 8) {
    regs_give<104>();
    const bool leader = elect_one();
    bool ok = true;
    uint32_t n_item = 0, n_step = 0, landed = 0;
    for (uint32_t round = 0; warp < (KV ? 11 : 10) && ok && round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t slot = w / per_slot, mine = w - slot * per_slot;
      const AttnTile t = attn_tile(p, slot, KV);
      if (!t.live) continue;
      const uint32_t tiles = (t.len + 127) / 128, steps = KV ? (tiles - t.tile) * p.group : t.tile + 1;
      // The heads and the tile that go past with a step.
      uint32_t head = KV ? mine * p.group : mine / p.group, at = KV ? t.tile : 0;
      auto next = [&]() {
        if (++at == tiles && KV) {
          at = t.tile;
          ++head;
        }
      };
      if (warp == 8) {
        ok = warp_wait(smem_u32(&s_stayempty), (n_item & 1) ^ 1, abort);
        if (!ok) break;
        if (leader) {
          const uint32_t bar = smem_u32(&s_stayfull);
          mbar_expect(bar, 2 * kTile);
          load_parts(stay, KV ? &maps.k : &maps.q, bar, mine, t.start + t.tile * 128, t.batch);
          load_parts(stay + kTile, KV ? &maps.v : &maps.go, bar, mine, t.start + t.tile * 128, t.batch);
        }
        __syncwarp();
        for (uint32_t i = 0; i < steps; ++i, ++n_step, next()) {
          ok = warp_wait(smem_u32(&s_empty), (n_step & 1) ^ 1, abort);
          if (!ok) break;
          const bool cut = p.offsets && (at + 1) * 128 > t.len;  // others' rows behind the sequence
          const uint32_t bar = cut ? smem_u32(&s_landed) : smem_u32(&s_full);
          if (leader) {
            mbar_expect(bar, 2 * kTile);
            load_parts(past, KV ? &maps.q : &maps.k, bar, head, t.start + at * 128, t.batch);
            load_parts(past + kTile, KV ? &maps.go : &maps.v, bar, head, t.start + at * 128, t.batch);
          }
          __syncwarp();
          if (cut) {
            ok = warp_wait(bar, landed & 1, abort);
            ++landed;
            if (!ok) break;
            at_clear(past, 2 * kParts, t.len - at * 128);
            if (leader) mbar_arrive(smem_u32(&s_full));
            __syncwarp();
          }
        }
      } else if (warp == 9) {
        ok = warp_wait(smem_u32(&s_stayfull), n_item & 1, abort);
        for (uint32_t i = 0; i < steps && ok; ++i, ++n_step) {
          ok = warp_wait(smem_u32(&s_full), n_step & 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            scores_of(tmem, stay, past);
            tc_commit<1>(smem_u32(&s_sfull));
            scores_of(tmem + kD, stay + kTile, past + kTile);
            tc_commit<1>(smem_u32(&s_dfull));
          }
          __syncwarp();
          if (i == 0) ok = warp_wait(smem_u32(&s_accempty), (n_item & 1) ^ 1, abort);
          if (KV) {
            ok = ok && warp_wait(smem_u32(&s_pfull), n_step & 1, abort);
            if (!ok) break;
            tc_fence_after();
            if (leader) sum_of(tmem + kAccP, tmem, tmem + kMoreP, past + kTile);
            __syncwarp();
          }
          ok = ok && warp_wait(smem_u32(&s_wfull), n_step & 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            sum_of(tmem + kAccW, tmem + kD, tmem + kMoreW, past);
            tc_commit<1>(smem_u32(&s_empty));
            if (i + 1 == steps) {
              tc_commit<1>(smem_u32(&s_accfull));
              tc_commit<1>(smem_u32(&s_stayempty));
            }
          }
          __syncwarp();
        }
      } else {
        for (uint32_t i = 0; i < steps; ++i, ++n_step, next()) {
          const uint32_t stage = n_step & 1;
          ok = warp_wait(smem_u32(&s_rempty[stage]), ((n_step / 2) & 1) ^ 1, abort);
          if (!ok) break;
          const int64_t rows = (int64_t(t.batch) * p.heads + head) * p.row_pitch + t.start + at * 128;
          const int64_t first = (int64_t(t.batch) * p.tokens + t.start + at * 128) * p.heads + head;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t r = lane + 32 * k;
            const bool in = at * 128 + r < t.len;  // behind the end the weight is 0
            s_rows[stage][r] = in ? -__ldcg(p.lse + first + int64_t(r) * p.heads) : -INFINITY;
            s_rows[stage][128 + r] = in ? -__ldcg(p.delta + rows + r) : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_rfull[stage]));
        }
      }
      ++n_item;
    }
  } else {
    regs_take<200>();
    const uint32_t half = warp >> 2, quad = warp & 3, own = quad * 32 + lane;
    const uint32_t lanes = tmem + (quad << 21);
    // KV: half 0 adds grad_v, half 1 grad_k, 64 columns each; else each 32 columns of grad_q.
    constexpr int kAcc = KV ? 64 : 32;
    const uint32_t acc_at = lanes + (KV ? (half ? kAccW : kAccP) : kAccW + half * 32);
    const F2 scale2 = f2_splat(p.scale), log2e = f2_splat(kLog2e);
    bool ok = true;
    uint32_t n_item = 0, n_step = 0;
    for (uint32_t round = 0; round * gridDim.x < items; ++round) {
      const uint32_t w = at_item(round);
      if (w >= items) continue;
      const uint32_t slot = w / per_slot, head = w - slot * per_slot;
      const AttnTile t = attn_tile(p, slot, KV);
      if (!t.live) continue;
      const uint32_t per = (t.len + 127) / 128 - t.tile, steps = KV ? per * p.group : t.tile + 1;
      const uint32_t row = t.tile * 128 + own;
      float lse = 0.f, delta = 0.f;
      if (!KV && row < t.len) {
        lse = -__ldcg(p.lse + (int64_t(t.batch) * p.tokens + t.start + row) * p.heads + head);
        delta = -__ldcg(p.delta + (int64_t(t.batch) * p.heads + head) * p.row_pitch + t.start + row);
      }
      float acc[kAcc];
#pragma unroll
      for (int j = 0; j < kAcc; ++j) acc[j] = 0.f;
      uint32_t q = 0;
      for (uint32_t i = 0; i < steps; ++i, ++n_step) {
        const uint32_t stage = n_step & 1;
        const float* rows = s_rows[stage] + half * 64;
        const bool diagonal = KV ? q == 0 : i + 1 == steps;
        if (KV) ok = ok && warp_wait(smem_u32(&s_rfull[stage]), (n_step / 2) & 1, abort);
        ok = ok && warp_wait(smem_u32(&s_sfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
        // The last step's sums: these scores come after them.
        if (i > 0) {
#pragma unroll
          for (int j = 0; j < kAcc; j += 32) add32(acc_at + j, acc + j);
        }
        float v[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* x = v + c * 32;
          read32(lanes + half * 64 + c * 32, x);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const F2 l = KV ? f2_pack(rows[c * 32 + j], rows[c * 32 + j + 1]) : f2_splat(lse);
            f2_unpack(f2_mul(f2_fma(f2_pack(x[j], x[j + 1]), scale2, l), log2e), x[j], x[j + 1]);
            x[j] = ex2(x[j]);
            x[j + 1] = ex2(x[j + 1]);
          }
          if (diagonal) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t col = half * 64 + c * 32 + j;
              if (KV ? col < own : col > own) x[j] = 0.f;
            }
          }
          if (KV) write_parts(lanes, lanes + kMoreP, half * 2 + c, x);
        }
        if (KV) {
          tc_wait_store();
          arrive_warp(smem_u32(&s_pfull));
        }
        ok = warp_wait(smem_u32(&s_dfull), n_step & 1, abort);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float d[32];
          read32(lanes + kD + half * 64 + c * 32, d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const F2 l = KV ? f2_pack(rows[128 + c * 32 + j], rows[128 + c * 32 + j + 1]) : f2_splat(delta);
            f2_unpack(f2_mul(f2_add(f2_pack(d[j], d[j + 1]), l), f2_pack(v[c * 32 + j], v[c * 32 + j + 1])), d[j], d[j + 1]);
          }
          if (diagonal) {  // a masked weight is 0 whatever the product is
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t col = half * 64 + c * 32 + j;
              if (KV ? col < own : col > own) d[j] = 0.f;
            }
          }
          write_parts(lanes + kD, lanes + kMoreW, half * 2 + c, d);
        }
        tc_wait_store();
        arrive_warp(smem_u32(&s_wfull));
        if (KV && lane == 0) mbar_arrive(smem_u32(&s_rempty[stage]));
        if (++q == per) q = 0;
      }
      ok = ok && warp_wait(smem_u32(&s_accfull), n_item & 1, abort);
      ++n_item;
      tc_fence_after();
      __syncwarp();
      const float by = ok ? (KV && half == 0 ? 1.f : p.scale) : qnan();
#pragma unroll
      for (int j = 0; j < kAcc; j += 32) add32(acc_at + j, acc + j);
      arrive_warp(smem_u32(&s_accempty));
#pragma unroll
      for (int j = 0; j < kAcc; ++j) acc[j] *= by;
      const AttnView& g = KV ? (half ? p.gk : p.gv) : p.gq;
      const bool wide = p.g_wide & (KV ? (half ? 2u : 4u) : 1u);
      if (row < t.len && g.p) {
        float* o = row_of(g, t, row, head);
#pragma unroll
        for (int j = 0; j < kAcc; j += 32) store_row_f32(o, g.elem, wide, acc + j, (KV ? 0 : half * 32) + j, p.dim);
      }
    }
  }
  __syncthreads();
  wait_in_flight(abort);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free<1>(tmem, 512);
  if (beside) pdl_wait();
}

template <typename K>
cudaError_t go(K k, uint32_t items, const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), int(kF32Smem));
  if (e != cudaSuccess) return e;
  return launch_k(k, items < kSms ? items : kSms, kF32Threads, kF32Smem, s, p, maps);
}

}  // namespace

cudaError_t launch_attn_split(int es, const AttnPlan& p, uint16_t* const* out, uint32_t count, uint32_t wide,
                              cudaStream_t s) {
  SplitPlan d{};
  const AttnView* x[4] = {&p.q, &p.k, &p.v, &p.go};
  d.count = count;
  d.tokens = p.tokens;
  d.dim = p.dim;
  d.wide = wide;
  d.beside = count == 4;
  for (uint32_t i = 0; i < count; ++i) {
    d.x[i] = *x[i];
    d.out[i] = out[i];
    d.heads[i] = i == 1 || i == 2 ? p.kv_heads : p.heads;
    d.first[i + 1] = d.first[i] + uint64_t(p.batch) * p.tokens * d.heads[i];
  }
  const uint32_t rows = kThreads / (p.dim <= 64 ? 8 : 16);  // of a CTA
  const unsigned cta = unsigned((d.first[count] + rows - 1) / rows);
  if (es == 4) return launch_k(k_attn_split<float, kParts, 64>, cta, kThreads, 0, s, d);
  return p.dim <= 64 ? launch_k(k_attn_split<__nv_bfloat16, 1, 64>, cta, kThreads, 0, s, d)
                     : launch_k(k_attn_split<__nv_bfloat16, 1, 128>, cta, kThreads, 0, s, d);
}

cudaError_t launch_attn_f32_fwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  return go(k_attn_f32_fwd, p.slots * p.heads, p, maps, s);
}

cudaError_t launch_attn_f32_bwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.want & 6) e = go(k_attn_f32_bwd<true>, p.slots * p.kv_heads, p, maps, s);
  if (e == cudaSuccess && (p.want & 1)) e = go(k_attn_f32_bwd<false>, p.slots * p.heads, p, maps, s);
  return e;
}

}  // namespace zr
