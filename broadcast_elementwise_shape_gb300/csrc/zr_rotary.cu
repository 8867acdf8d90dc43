// zr_rotary.cu — rotary positions: kernels, plan and C entry points.
//
// A head's pair (i, k) is turned by the angle position * rate.  The rate is
// kept as turns a position in 64-bit fixed point, so that position * rate
// modulo 2^64 is the angle as a fraction of a turn: whole turns fall off the
// top, and a far position costs no accuracy (in binary32 the product alone would be
// off by 0.06 rad at position 2^20).  The nearest quarter turn is taken off in
// the integer, the rest, at most an eighth of a turn, goes through sine and cosine in binary32.
// The backward is the turn by the negative angle.
//
// Bound by HBM: each element is read and written once.  The angles are the same
// for all heads of a token, so a CTA computes those of its tokens once, into
// shared memory, and streams the heads past them: bf16 [65536, 40, 128] 201 us,
// 6.7 TB/s.  Heads of odd sizes go element by element, at 1.6 to 1.8 TB/s in bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "zr_checks.h"
#include "zr_kernels.cuh"
#include "zr_launch.h"

namespace zr {

// Slots: 0 x, 1 positions, 3 out.
struct RotPlan {
  const void* x;
  const void* positions;     // or null
  void* out;
  int64_t start;
  Decomp lead;               // a token's offsets
  FastDiv last;              // without positions: size of the last leading dim
  FastDiv per_token;         // items of a token
  FastDiv per_head;          // places of a head
  uint32_t heads, share;     // heads; of an item
  int64_t head[2];           // stride of a head: x, out
  int64_t inner[2];          // of an element (element-wise plans)
  uint32_t tokens, tile;     // tokens in all; per CTA
  uint32_t pairs;
  uint32_t turned;           // places of a head that turn; those behind pass through
  uint32_t i64, interleaved, backward;
  float magnitude;
  uint64_t turns[ZR_ROTARY_PAIRS];
};

namespace {

constexpr uint32_t kRotAngles = 2048;  // (cos, sin) of a tile, 16 KB
constexpr int kRotHeads = 4;

__device__ __forceinline__ float2 rot_angle(const RotPlan& p, int64_t position, uint32_t pair) {
  const uint64_t turn = uint64_t(position) * p.turns[pair];
  const int32_t a = int32_t(turn >> 32);                    // 2^-32 of a turn
  const uint32_t quarter = (uint32_t(a) + (1u << 29)) >> 30;
  const int32_t rest = int32_t(uint32_t(a) - (quarter << 30));
  float s, c;
  sincospif(float(rest) * 0x1p-31f, &s, &c);                // |rest| <= an eighth of a turn
  const float cq = quarter & 1 ? -s : c, sq = quarter & 1 ? c : s;
  const float m = quarter & 2 ? -p.magnitude : p.magnitude;
  return make_float2(m * cq, (p.backward ? -m : m) * sq);
}

__device__ __forceinline__ void rot_turn(float& a, float& b, float2 t) {
  const float u = __fmaf_rn(a, t.x, -(b * t.y));
  b = __fmaf_rn(b, t.x, a * t.y);
  a = u;
}

template <typename E, int V>
struct RotVec {
  float v[V];
  __device__ __forceinline__ void unpack(uint4 w) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (V == 4) v[i] = __uint_as_float(r[i]);
      else v[i] = __uint_as_float(i & 1 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
    }
  }
  __device__ __forceinline__ uint4 pack() const {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 4) {
        r[i] = __float_as_uint(v[i]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

// An item is a place in the head and a group of up to kRotHeads heads: its angles
// are read from shared memory once, and nothing but an addition lies between one
// head and the next.  WIDE: the place is 16 bytes of neighbouring pairs (half
// layout: 16 bytes of each half), V elements.  Otherwise one pair, or one element
// that passes through.
template <typename E, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ RotPlan p) {
  constexpr int V = WIDE ? 16 / int(sizeof(E)) : 1;
  constexpr int A = WIDE ? V : 1;           // angles of an item, at most
  extern __shared__ float2 s_angle[];       // [token][pair]
  __shared__ int64_t s_at[2 * 32];
  pdl_trigger();
  const uint32_t first = blockIdx.x * p.tile;
  const uint32_t n = p.tokens - first < p.tile ? p.tokens - first : p.tile;
  pdl_wait();
  if (threadIdx.x < n) {
    int64_t off[kMaxOperands];
    decomp_offsets(p.lead, first + threadIdx.x, off);
    s_at[2 * threadIdx.x] = off[0];
    s_at[2 * threadIdx.x + 1] = off[kSlotOut];
  }
  for (uint32_t i = threadIdx.x; i < n * p.pairs; i += kThreads) {
    const uint32_t t = i / p.pairs, pair = i - t * p.pairs, token = first + t;
    int64_t position;
    if (p.positions) {
      int64_t off[kMaxOperands];
      decomp_offsets(p.lead, token, off);
      position = p.i64 ? static_cast<const int64_t*>(p.positions)[off[1]]
                       : int64_t(static_cast<const int32_t*>(p.positions)[off[1]]);
    } else {
      position = int64_t(token - fd_div(p.last, token) * p.last.d);
    }
    s_angle[i] = rot_angle(p, position + p.start, pair);
  }
  __syncthreads();
  const uint32_t total = n * p.per_token.d;
  for (uint32_t i = threadIdx.x; i < total; i += kThreads) {
    const uint32_t t = fd_div(p.per_token, i), j = i - t * p.per_token.d;
    const uint32_t group = fd_div(p.per_head, j), k = j - group * p.per_head.d;
    const uint32_t h0 = group * p.share, heads = p.heads - h0 < p.share ? p.heads - h0 : p.share;
    const bool turn = k < p.turned;
    const uint32_t e = WIDE ? (turn || p.interleaved ? k * V : 2 * p.pairs + (k - p.turned) * V)
                            : (turn ? (p.interleaved ? 2 * k : k) : p.pairs + k);
    const uint32_t apart = p.interleaved ? 1 : p.pairs;  // from a pair's first element to its second
    const int64_t si = WIDE ? 1 : p.inner[0], so = WIDE ? 1 : p.inner[1];
    const E* x = static_cast<const E*>(p.x) + s_at[2 * t] + int64_t(h0) * p.head[0] + int64_t(e) * si;
    E* out = static_cast<E*>(p.out) + s_at[2 * t + 1] + int64_t(h0) * p.head[1] + int64_t(e) * so;
    float2 angle[A];
    if (turn) {
      const float2* from = s_angle + t * p.pairs + (WIDE ? (p.interleaved ? k * (V / 2) : k * V) : k);
#pragma unroll
      for (int a = 0; a < A; ++a)
        if (!WIDE || a < V / 2 || !p.interleaved) angle[a] = from[a];
    }
    uint4 w[kRotHeads][2];
    float f[kRotHeads][2];
    const bool both = turn && (!WIDE || !p.interleaved);
#pragma unroll
    for (int u = 0; u < kRotHeads; ++u) {
      if (uint32_t(u) >= heads) continue;
      const E* from = x + u * p.head[0];
      if constexpr (WIDE) {
        w[u][0] = *reinterpret_cast<const uint4*>(from);
        if (both) w[u][1] = *reinterpret_cast<const uint4*>(from + apart);
      } else {
        f[u][0] = ld1(from, false);
        if (both) f[u][1] = ld1(from + apart * si, false);
      }
    }
#pragma unroll
    for (int u = 0; u < kRotHeads; ++u) {
      if (uint32_t(u) >= heads) continue;
      E* to = out + u * p.head[1];
      if constexpr (WIDE) {
        RotVec<E, V> a, b;
        if (both) {
          a.unpack(w[u][0]);
          b.unpack(w[u][1]);
#pragma unroll
          for (int v = 0; v < V; ++v) rot_turn(a.v[v], b.v[v], angle[v]);
          *reinterpret_cast<uint4*>(to + apart) = b.pack();
          w[u][0] = a.pack();
        } else if (turn) {
          a.unpack(w[u][0]);
#pragma unroll
          for (int v = 0; v < V / 2; ++v) rot_turn(a.v[2 * v], a.v[2 * v + 1], angle[v]);
          w[u][0] = a.pack();
        }
        *reinterpret_cast<uint4*>(to) = w[u][0];
      } else {
        if (both) {
          rot_turn(f[u][0], f[u][1], angle[0]);
          st1(to + apart * so, f[u][1]);
        }
        st1(to, f[u][0]);
      }
    }
  }
}

struct RotSet {
  RotPlan p;
  TDesc x, pos, out;
  int es = 4;
  bool empty = false, wide = false;
  uint32_t n_cta = 0;
};

int plan_rotary(zr_dtype dtype, const zr_tensor& x, const zr_rotary* plan, zr_index type,
                const zr_tensor& positions, int64_t start, void* out, const int64_t* out_strides,
                bool backward, RotSet* S) {
  if (!plan) return ZR_ERR_NULL;
  if (dtype != ZR_F32 && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  if (type != ZR_I32 && type != ZR_I64) return ZR_ERR_DTYPE;
  if (plan->part < 2 || plan->part > 2 * ZR_ROTARY_PAIRS || plan->part % 2) return ZR_ERR_SIZE;
  S->es = dtype == ZR_BF16 ? 2 : 4;
  RotPlan& p = S->p;
  p = RotPlan{};
  int rc = read_tensor(x, &S->x);
  if (rc) return rc;
  const int n = S->x.nd;
  if (n < 2) return ZR_ERR_RANK;
  if (S->x.size[n - 1] < plan->part) return ZR_ERR_SHAPE;
  if ((rc = read_tensor(zr_tensor{out, n, S->x.size, out_strides}, &S->out))) return rc;
  const bool given = positions.data != nullptr;
  S->pos = TDesc{};
  if (given) {
    if ((rc = read_tensor(positions, &S->pos))) return rc;
    if (S->pos.nd != n - 2) return ZR_ERR_SHAPE;
    for (int d = 0; d + 2 < n; ++d)
      if (S->pos.size[d] != S->x.size[d]) return ZR_ERR_SHAPE;
  }
  if (S->x.numel == 0) {
    S->empty = true;
    return ZR_OK;
  }
  if (!S->x.ptr || !out) return ZR_ERR_NULL;
  if (!non_overlapping(S->out)) return ZR_ERR_LAYOUT;
  const Span so = span_of(out, S->out.extent, S->es);
  if (overlaps(so, span_of(S->x.ptr, S->x.extent, S->es)) && !same_layout(S->x, S->out))
    return ZR_ERR_LAYOUT;
  const int ps = type == ZR_I64 ? 8 : 4;
  if (given && reinterpret_cast<uintptr_t>(positions.data) % ps) return ZR_ERR_LAYOUT;
  if (overlaps(so, span_of(positions.data, S->pos.extent, ps))) return ZR_ERR_LAYOUT;

  const int64_t H = S->x.size[n - 2], D = S->x.size[n - 1];
  if (H >= (int64_t(1) << 20) || D >= (int64_t(1) << 20)) return ZR_ERR_SIZE;
  int64_t tokens = 1, st[kProbSlots][kMaxDims] = {};
  for (int d = 0; d + 2 < n; ++d) {
    if (S->x.size[d] >= (int64_t(1) << 31) / tokens) return ZR_ERR_SIZE;
    tokens *= S->x.size[d];
    st[0][d] = S->x.stride[d];
    st[1][d] = given ? S->pos.stride[d] : 0;
    st[kSlotOut][d] = S->out.stride[d];
  }
  Prob P;
  const uint32_t slots = 1u | (given ? 2u : 0u) | (1u << kSlotOut);
  if (n > 2) {
    if ((rc = coalesce(n - 2, S->x.size, st, slots, -1, &P))) return rc;
    p.lead.n = P.n;
    for (int i = 0; i < P.n; ++i) {
      const int d = P.n - 1 - i;
      p.lead.div[i] = make_fastdiv(uint32_t(P.size[d]));
      for (int k = 0; k < kMaxOperands; ++k) p.lead.stride[k][i] = P.st[k][d];
    }
  }
  p.x = S->x.ptr;
  p.positions = positions.data;
  p.out = out;
  p.start = start;
  p.last = make_fastdiv(n > 2 ? uint32_t(S->x.size[n - 3]) : 1);
  p.head[0] = S->x.stride[n - 2];
  p.head[1] = S->out.stride[n - 2];
  p.inner[0] = S->x.stride[n - 1];
  p.inner[1] = S->out.stride[n - 1];
  p.tokens = uint32_t(tokens);
  p.pairs = uint32_t(plan->part) / 2;
  p.i64 = type == ZR_I64;
  p.interleaved = plan->interleaved != 0;
  p.backward = backward;
  p.magnitude = plan->magnitude;
  std::copy(plan->turns, plan->turns + p.pairs, p.turns);

  const int V = 16 / S->es;
  bool wide = p.inner[0] == 1 && p.inner[1] == 1 && D % V == 0 && plan->part % V == 0 &&
              (p.interleaved || p.pairs % uint32_t(V) == 0);
  for (int k = 0; k < 2; ++k) {
    if (reinterpret_cast<uintptr_t>(k ? out : S->x.ptr) % 16) wide = false;
    const TDesc& t = k ? S->out : S->x;
    for (int d = 0; d + 1 < n; ++d)
      if (t.size[d] > 1 && t.stride[d] % V) wide = false;
  }
  S->wide = wide;
  const uint32_t v = wide ? uint32_t(V) : 1;
  p.turned = wide ? (p.interleaved ? uint32_t(plan->part) : p.pairs) / v : p.pairs;
  const uint32_t per_head = p.turned + uint32_t(D - plan->part) / v;
  if (uint64_t(per_head) * uint64_t(H) >= (uint64_t(1) << 26)) return ZR_ERR_SIZE;
  // Heads of an item: one where there are few items, for latency, up to four, so
  // that a thread has that many loads under way and reads its angles once.
  p.heads = uint32_t(H);
  const uint64_t items = uint64_t(per_head) * uint64_t(H) * p.tokens;
  p.share = uint32_t(std::min<uint64_t>(kRotHeads, 1 + items / (kSms * 2 * kThreads)));
  p.per_head = make_fastdiv(per_head);
  p.per_token = make_fastdiv(per_head * ((p.heads + p.share - 1) / p.share));
  // Tokens of a CTA: two items a thread, but no fewer CTAs than four a SM, at most
  // 32 tokens, and their angles in 16 KB.
  uint32_t tile = (2 * kThreads + p.per_token.d - 1) / p.per_token.d;
  tile = std::min({tile, 32u, kRotAngles / p.pairs, std::max(1u, p.tokens / (4 * kSms))});
  p.tile = std::max(1u, tile);
  S->n_cta = (p.tokens + p.tile - 1) / p.tile;
  return ZR_OK;
}

int run_rotary(const char* name, zr_dtype dtype, const zr_tensor& x, const zr_rotary* plan,
               zr_index type, const zr_tensor& positions, int64_t start, void* out,
               const int64_t* out_strides, bool backward, zr_stream_t stream) {
  RotSet S;
  int rc = plan_rotary(dtype, x, plan, type, positions, start, out, out_strides, backward, &S);
  if (rc || S.empty) return rc;
  const RotPlan& p = S.p;
  trace(name, [&] {
    return std::string("{\"kernel\":\"rotary\",\"wide\":") + (S.wide ? "true" : "false") +
           ",\"tile\":" + std::to_string(p.tile) + ",\"n_cta\":" + std::to_string(S.n_cta) + "}";
  });
  for (const void* q : {p.x, p.positions, static_cast<const void*>(out)})
    if (q && (rc = check_device_ptr(q))) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t smem = size_t(p.tile) * p.pairs * sizeof(float2);
  const auto k = S.es == 2 ? (S.wide ? k_rotary<__nv_bfloat16, true> : k_rotary<__nv_bfloat16, false>)
                           : (S.wide ? k_rotary<float, true> : k_rotary<float, false>);
  return cuda_status(launch_k(k, S.n_cta, kThreads, smem, st, p));
}

}  // namespace
}  // namespace zr

extern "C" {

int zr_rotary_plan(int32_t part, int32_t interleaved, double base, double factor, double original,
                   double low, double high, double magnitude, zr_rotary* plan) {
  if (!plan) return ZR_ERR_NULL;
  if (part < 2 || part > 2 * ZR_ROTARY_PAIRS || part % 2) return ZR_ERR_SIZE;
  if (!(base >= 1) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) ||
      !(original >= 0) || !std::isfinite(original) || !std::isfinite(magnitude) ||
      (original > 0 && (!(low >= 0) || !(high > low) || !std::isfinite(high))))
    return ZR_ERR_VALUE;
  *plan = zr_rotary{};
  plan->part = part;
  plan->interleaved = interleaved != 0;
  plan->magnitude = float(magnitude);
  const double two_pi = 6.283185307179586;
  for (int j = 0; j < part / 2; ++j) {
    double rate = std::pow(base, -2.0 * j / part);
    if (original > 0) {
      const double w = std::min(1.0, std::max(0.0, (original * rate / two_pi - low) / (high - low)));
      rate *= w + (1 - w) / factor;
    } else {
      rate /= factor;
    }
    const double turn = rate / two_pi;
    const double t = std::nearbyint(std::ldexp(turn - std::floor(turn), 64));
    plan->turns[j] = t < 0x1p64 ? uint64_t(t) : 0;
  }
  return ZR_OK;
}

int zr_rotary_fwd(zr_dtype dtype, zr_tensor x, const zr_rotary* plan, zr_index position_type,
                  zr_tensor positions, int64_t start, void* out, const int64_t* out_strides,
                  zr_stream_t stream) {
  return zr::run_rotary("zr_rotary_fwd", dtype, x, plan, position_type, positions, start, out,
                        out_strides, false, stream);
}

int zr_rotary_bwd(zr_dtype dtype, zr_tensor grad_out, const zr_rotary* plan, zr_index position_type,
                  zr_tensor positions, int64_t start, void* grad_x, const int64_t* grad_x_strides,
                  zr_stream_t stream) {
  return zr::run_rotary("zr_rotary_bwd", dtype, grad_out, plan, position_type, positions, start,
                        grad_x, grad_x_strides, true, stream);
}

}  // extern "C"
