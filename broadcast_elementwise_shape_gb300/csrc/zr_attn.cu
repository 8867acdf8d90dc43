// zr_attn.cu — causal attention: plan and C entry points.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "zr_attn.h"
#include "zr_checks.h"
#include "zr_launch.h"
#include "zr_maps.h"

namespace zr {
namespace {

constexpr float kLog2eHost = 1.4426950408889634f;

struct AttnSet {
  AttnPlan p;
  TDesc q, k, v, o, go, gq, gk, gv;
  int es = 4;
  bool empty = false;
  size_t ws = 0;
};

AttnView view_of(const TDesc& t) {
  const int n = t.nd;
  return {t.ptr, n == 4 ? t.stride[0] : 0, t.stride[n - 3], t.stride[n - 2], t.stride[n - 1]};
}

// Everything that both directions share.  Leaves S->empty where there is
// nothing to do.
int plan_attn(zr_dtype dtype, const zr_tensor& q, const zr_tensor& k, const zr_tensor& v, float scale,
              const int32_t* offsets, int32_t sequences, AttnSet* S) {
  if (dtype != ZR_F32 && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  S->es = dtype == ZR_BF16 ? 2 : 4;
  AttnPlan& p = S->p;
  p = AttnPlan{};
  int rc;
  if ((rc = read_tensor(q, &S->q)) || (rc = read_tensor(k, &S->k)) || (rc = read_tensor(v, &S->v))) return rc;
  const int n = S->q.nd;
  if (n < 3 || n > 4 || S->k.nd != n || S->v.nd != n) return ZR_ERR_RANK;
  if (offsets && n != 3) return ZR_ERR_RANK;
  if (sequences < 0) return ZR_ERR_SIZE;
  if (!std::isfinite(scale)) return ZR_ERR_VALUE;
  const int64_t* sq = S->q.size;
  for (int d = 0; d < n; ++d) {
    if (S->k.size[d] != S->v.size[d]) return ZR_ERR_SHAPE;
    if (d != n - 2 && S->k.size[d] != sq[d]) return ZR_ERR_SHAPE;
  }
  const int64_t B = n == 4 ? sq[0] : 1, T = sq[n - 3], H = sq[n - 2], K = S->k.size[n - 2], D = sq[n - 1];
  if (H < 1 || K < 1 || H % K != 0 || D < 1) return ZR_ERR_SHAPE;
  if (D > 256) return ZR_ERR_SIZE;
  if (reinterpret_cast<uintptr_t>(offsets) % 4) return ZR_ERR_LAYOUT;
  if (B == 0 || T == 0 || (offsets && sequences == 0)) {
    S->empty = true;
    return ZR_OK;
  }
  // Rows (batch, token, head) and tiles are counted in 31 bits.
  if (T >= (int64_t(1) << 30) || H >= (int64_t(1) << 20) || B >= (int64_t(1) << 30) ||
      B * H >= (int64_t(1) << 31) || (T + 127) / 128 * 128 >= (int64_t(1) << 31) / (B * H))
    return ZR_ERR_SIZE;
  const int64_t tiles = offsets ? T / 64 + std::min<int64_t>(sequences, T) : (T + 63) / 64 * B;
  if (tiles >= (int64_t(1) << 31) / H) return ZR_ERR_SIZE;
  p.offsets = offsets;
  p.sequences = uint32_t(sequences);
  p.batch = uint32_t(B);
  p.tokens = uint32_t(T);
  p.heads = uint32_t(H);
  p.kv_heads = uint32_t(K);
  p.group = uint32_t(H / K);
  p.dim = uint32_t(D);
  p.row_pitch = uint32_t((T + 127) / 128 * 128);
  p.tile_rows = 64;
  p.slots = uint32_t(tiles);
  p.scale = scale;
  p.scale_log2 = scale * kLog2eHost;
  p.q = view_of(S->q);
  p.k = view_of(S->k);
  p.v = view_of(S->v);
  return ZR_OK;
}

// A written tensor of `like`'s shape.
int plan_out(const TDesc& like, void* data, const int64_t* strides, TDesc* t) {
  const int rc = read_tensor(zr_tensor{data, like.nd, like.size, strides}, t);
  if (rc) return rc;
  return data && !non_overlapping(*t) ? ZR_ERR_LAYOUT : ZR_OK;
}

// 16-byte accesses along the elements.
bool wide(const TDesc& t, int es) {
  const int n = t.nd;
  if (!t.ptr) return true;
  if (t.size[n - 1] * es % 16 != 0 || (t.size[n - 1] > 1 && t.stride[n - 1] != 1)) return false;
  if (reinterpret_cast<uintptr_t>(t.ptr) % 16) return false;
  for (int d = 0; d + 1 < n; ++d)
    if (t.size[d] > 1 && t.stride[d] * es % 16) return false;
  return true;
}

// Whether two tensors whose spans meet share no element: both have unit
// elements and the same batch and token strides, and within a token's stride
// their heads lie in separate runs, as the parts of a projection's rows do.
bool interleaved(const TDesc& x, const TDesc& y, int es) {
  const int n = x.nd;
  int64_t run[2], pitch = 0;  // a token's run; tokens are at least this far apart
  const TDesc* t[2] = {&x, &y};
  for (int i = 0; i < 2; ++i) {
    const TDesc& a = *t[i];
    if (a.size[n - 1] > 1 && a.stride[n - 1] != 1) return false;
    if (a.size[n - 2] > 1 && a.stride[n - 2] < a.size[n - 1]) return false;
    run[i] = (a.size[n - 2] - 1) * a.stride[n - 2] + a.size[n - 1];
  }
  for (int d = 0; d + 2 < n; ++d) {
    if (x.size[d] <= 1) continue;
    if (x.stride[d] != y.stride[d]) return false;
    pitch = pitch ? std::min(pitch, x.stride[d]) : x.stride[d];
    // Every other leading dim's stride is a multiple of the smallest.
  }
  if (!pitch) return false;
  for (int d = 0; d + 2 < n; ++d)
    if (x.size[d] > 1 && x.stride[d] % pitch) return false;
  const int64_t apart = int64_t(reinterpret_cast<intptr_t>(y.ptr) - reinterpret_cast<intptr_t>(x.ptr));
  if (apart % es) return false;
  // Offsets of a token's run modulo the pitch: [0, run x) and [at, at + run y).
  const int64_t at = ((apart / es) % pitch + pitch) % pitch;
  return run[0] <= at && at + run[1] <= pitch;
}

// No written buffer may overlap another, or an input.
int check_overlaps(const Span* in, int n_in, const Span* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i], in[j])) return ZR_ERR_LAYOUT;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return ZR_ERR_LAYOUT;
  }
  return ZR_OK;
}

// What the tensor-core kernels read by TMA: unit elements, rows that start on 16
// bytes and whose strides are positive multiples of them.
bool mappable(const TDesc& t, int es) {
  if (!wide(t, es)) return false;
  for (int d = 0; d + 1 < t.nd; ++d)
    if (t.size[d] > 1 && (t.stride[d] <= 0 || t.stride[d] * es >= (int64_t(1) << 40))) return false;
  return true;
}
// The tensor cores take bfloat16 heads of up to 128 elements, and binary32 ones
// of up to 64 in parts (zr_attn_f32.cu), with a positive scale: a row's maximum is that
// of its products.  Up to 64 tokens the copy into parts costs more than it gains: [64, 64]
// tokens of 12 heads of 64, forward 53 us, by multiply-adds 36; [4, 128] 13.8 and 20.9.
bool tensor_cores(const AttnSet& S, float scale) {
  return scale > 0 && (S.es == 2 ? S.p.dim <= 128 : S.p.dim <= 64 && S.p.tokens > 64);
}
// Whether the operands are copied for it: binary32 always (into parts), bfloat16
// rows that no tensor map describes (odd addresses, head sizes or strides): [2048]
// tokens of 16 heads of 81, 88 us with their copy.
bool copied(const AttnSet& S, bool backward) {
  return S.es == 4 || !mappable(S.q, 2) || !mappable(S.k, 2) || !mappable(S.v, 2) || (backward && !mappable(S.go, 2));
}
// Boxes of 64 elements x 128 tokens; what is out of range reads as zero.
bool tile_map(CUtensorMap* m, const TDesc& t) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const int n = t.nd;
  const auto stride = [&](int d) { return cuuint64_t(t.size[d] > 1 ? t.stride[d] * 2 : 16); };
  const cuuint64_t dims[4] = {cuuint64_t(t.size[n - 1]), cuuint64_t(t.size[n - 2]), cuuint64_t(t.size[n - 3]),
                              cuuint64_t(n == 4 ? t.size[0] : 1)};
  const cuuint64_t strides[3] = {stride(n - 2), stride(n - 3), n == 4 ? stride(0) : 16};
  const cuuint32_t box[4] = {64, 1, 128, 1}, step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<float*>(t.ptr), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The copies of q, k, v and (count 4) grad_out behind `at` bytes of workspace.
struct Copies {
  uint64_t rows[4];
  size_t at[4], end;
};
Copies copies_of(const AttnSet& S, int count, size_t at) {
  const AttnPlan& p = S.p;
  Copies x{};
  const size_t row = S.es == 4 ? 3 * 128 : p.dim <= 64 ? 128 : 256;  // bytes
  for (int i = 0; i < count; ++i) {
    x.rows[i] = uint64_t(p.batch) * p.tokens * (i == 1 || i == 2 ? p.kv_heads : p.heads);
    x.at[i] = at = (at + 255) / 256 * 256;
    at += size_t(x.rows[i]) * row;
  }
  x.end = at;
  return x;
}
// Boxes of 64 elements of 128 tokens, all parts of binary32 ones.
bool copy_map(CUtensorMap* m, const AttnSet& S, void* base, uint64_t rows, uint32_t heads) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const AttnPlan& p = S.p;
  const cuuint32_t parts = S.es == 4 ? 3 : 1;
  const cuuint64_t width = p.dim <= 64 ? 64 : 128, token = heads * width * 2;
  const cuuint64_t dims[5] = {width, heads, p.tokens, p.batch, parts};
  const cuuint64_t strides[4] = {width * 2, token, token * p.tokens, cuuint64_t(rows) * width * 2};
  const cuuint32_t box[5] = {64, 1, 128, 1, parts}, step[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, parts == 3 ? 5 : 4, base, dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The kernels' maps, over the operands or over their copies, which this makes.
cudaError_t operands(const AttnSet& S, bool copy, const Copies& x, int count, void* workspace, AttnMaps* maps, cudaStream_t s) {
  const AttnPlan& p = S.p;
  CUtensorMap* m[4] = {&maps->q, &maps->k, &maps->v, &maps->go};
  const TDesc* t[4] = {&S.q, &S.k, &S.v, &S.go};
  uint16_t* out[4] = {};
  uint32_t w = 0;
  for (int i = 0; i < count; ++i) {
    if (!copy) {
      if (!tile_map(m[i], *t[i])) return cudaErrorInvalidValue;
      continue;
    }
    out[i] = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + x.at[i]);
    if (!copy_map(m[i], S, out[i], x.rows[i], i == 1 || i == 2 ? p.kv_heads : p.heads)) return cudaErrorInvalidValue;
    if (wide(*t[i], S.es)) w |= 1u << i;
  }
  if (count == 3) maps->go = maps->q;
  return copy ? launch_attn_split(S.es, p, out, uint32_t(count), w, s) : cudaSuccess;
}
// Tiles of `rows` rows.
void set_tiles(AttnPlan* p, uint32_t rows) {
  p->tile_rows = rows;
  p->slots = p->offsets ? p->tokens / rows + (p->sequences < p->tokens ? p->sequences : p->tokens)
                        : (p->tokens + rows - 1) / rows * p->batch;
}

// Shares of a key tile's steps in the backward (bfloat16 on the tensor cores).
// Tiles are dealt out whole, heaviest first, which evens out with some three tiles
// for each SM; with fewer (few key heads, short batches) each is cut, up to
// eight times, and the shares' sums are added at the end: [1, 4096], 8 heads on one key head, D =
// 128, grad_k and grad_v 328 us in one share.  A share has four steps of the average tile at least.
uint32_t shares(const AttnPlan& p) {
  const uint64_t tiles = (uint64_t(p.tokens) + 127) / 128, items = tiles * p.batch * p.kv_heads;
  const uint64_t average = std::max<uint64_t>(1, (tiles + 1) / 2 * p.group);
  return uint32_t(std::max<uint64_t>(1, std::min<uint64_t>({8, 3 * kSms / items, average / 4})));
}

const char* kernel_name(bool tc, bool copy, int es) { return !tc ? "any" : es == 4 ? "parts" : copy ? "copied" : "tensor"; }

// The forward's pairs of query tiles likewise, along their keys; a share has
// eight key tiles of the average pair at least.
uint32_t fwd_shares(const AttnPlan& p) {
  const uint64_t tiles = (uint64_t(p.tokens) + 255) / 256, items = tiles * p.batch * p.heads;
  return uint32_t(std::max<uint64_t>(1, std::min<uint64_t>({8, 3 * kSms / items, (tiles + 1) / 8})));
}

std::string plan_json(const AttnSet& S, const char* kernel) {
  const AttnPlan& p = S.p;
  return std::string("{\"kernel\":\"") + kernel + "\",\"tile\":" + std::to_string(p.tile_rows) +
         ",\"slots\":" + std::to_string(p.slots) + ",\"dim\":" + std::to_string(p.dim) +
         ",\"workspace\":" + std::to_string(S.ws) + "}";
}

int fwd_impl(zr_dtype dtype, const zr_tensor& q, const zr_tensor& k, const zr_tensor& v, float scale,
             const int32_t* offsets, int32_t sequences, void* out, const int64_t* out_strides, void* low,
             float* lse, void* workspace, size_t* workspace_bytes, zr_stream_t stream) {
  if (!workspace_bytes) return ZR_ERR_NULL;
  AttnSet S;
  int rc = plan_attn(dtype, q, k, v, scale, offsets, sequences, &S);
  if (rc) return rc;
  if ((rc = plan_out(S.q, out, out_strides, &S.o))) return rc;
  if (low && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  const bool tc = !S.empty && tensor_cores(S, scale), copy = tc && copied(S, false);
  const Copies copies = copy ? copies_of(S, 3, 0) : Copies{};
  S.ws = copies.end;
  S.p.splits = tc && S.es == 2 ? fwd_shares(S.p) : 1;
  const size_t part_at = (S.ws + 255) / 256 * 256;
  if (S.p.splits > 1)
    S.ws = part_at + size_t(S.p.splits) * S.p.batch * S.p.tokens * S.p.heads * ((S.p.dim <= 64 ? 64 : 128) + 1) * sizeof(float);
  if (!workspace) {
    *workspace_bytes = S.ws;
    return ZR_OK;
  }
  if (S.empty) return ZR_OK;
  if (!S.q.ptr || !S.k.ptr || !S.v.ptr || !out) return ZR_ERR_NULL;
  if (*workspace_bytes < S.ws || reinterpret_cast<uintptr_t>(workspace) % 16) return ZR_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(low) % S.es || reinterpret_cast<uintptr_t>(lse) % 4) return ZR_ERR_LAYOUT;
  AttnPlan& p = S.p;
  const Span in[] = {span_of(S.q.ptr, S.q.extent, S.es), span_of(S.k.ptr, S.k.extent, S.es),
                     span_of(S.v.ptr, S.v.extent, S.es), span_of(offsets, int64_t(sequences) + 1, 4)};
  const Span outs[] = {span_of(out, S.o.extent, S.es), span_of(low, S.q.numel, S.es),
                       span_of(lse, S.q.numel / p.dim, 4), span_of(workspace, int64_t(S.ws), 1)};
  if ((rc = check_overlaps(in, 4, outs, 4))) return rc;
  p.o = view_of(S.o);
  p.low = low;
  p.lse = lse;
  p.vec = wide(S.q, S.es) && wide(S.k, S.es) && wide(S.v, S.es);
  p.o_wide = wide(S.o, S.es);
  p.low_wide = reinterpret_cast<uintptr_t>(low) % 16 == 0 && p.dim % 8 == 0;
  if (tc) set_tiles(&p, 256);
  p.part = p.splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_at) : nullptr;
  trace("zr_attention_fwd", [&] { return plan_json(S, kernel_name(tc, copy, S.es)); });
  for (const void* x : {p.q.p, p.k.p, p.v.p, static_cast<const void*>(out), static_cast<const void*>(low),
                        static_cast<const void*>(lse), static_cast<const void*>(offsets),
                        static_cast<const void*>(S.ws ? workspace : nullptr)})
    if (x && (rc = check_device_ptr(x))) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!tc) return cuda_status(launch_attn_any_fwd(S.es, p, st));
  AttnMaps maps;
  const cudaError_t e = operands(S, copy, copies, 3, workspace, &maps, st);
  if (e != cudaSuccess) return ZR_ERR_CUDA;
  return cuda_status(S.es == 4 ? launch_attn_f32_fwd(p, maps, st) : launch_attn_fwd(p, maps, st));
}

int bwd_impl(zr_dtype dtype, const zr_tensor& grad_out, const zr_tensor& q, const zr_tensor& k,
             const zr_tensor& v, const zr_tensor& out, const void* low, const float* lse, float scale,
             const int32_t* offsets, int32_t sequences, void* grad_q, const int64_t* grad_q_strides,
             void* grad_k, const int64_t* grad_k_strides, void* grad_v, const int64_t* grad_v_strides,
             void* workspace, size_t* workspace_bytes, zr_stream_t stream) {
  if (!workspace_bytes) return ZR_ERR_NULL;
  AttnSet S;
  int rc = plan_attn(dtype, q, k, v, scale, offsets, sequences, &S);
  if (rc) return rc;
  if ((rc = read_tensor(grad_out, &S.go)) || (rc = read_tensor(out, &S.o))) return rc;
  for (const TDesc* t : {&S.go, &S.o}) {
    if (t->nd != S.q.nd) return ZR_ERR_RANK;
    for (int d = 0; d < t->nd; ++d)
      if (t->size[d] != S.q.size[d]) return ZR_ERR_SHAPE;
  }
  if ((rc = plan_out(S.q, grad_q, grad_q_strides, &S.gq)) || (rc = plan_out(S.k, grad_k, grad_k_strides, &S.gk)) ||
      (rc = plan_out(S.v, grad_v, grad_v_strides, &S.gv)))
    return rc;
  if (low && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  AttnPlan& p = S.p;
  const size_t rows = S.empty ? 0 : size_t(p.batch) * p.heads * p.row_pitch;
  const bool tc = !S.empty && tensor_cores(S, scale), copy = tc && copied(S, true);
  const Copies copies = copy ? copies_of(S, 4, 2 * rows * sizeof(float)) : Copies{};
  S.ws = copy ? copies.end : 2 * rows * sizeof(float);
  p.splits = tc && S.es == 2 && (grad_k || grad_v) ? shares(p) : 1;
  const size_t part_at = (S.ws + 255) / 256 * 256;
  if (p.splits > 1)
    S.ws = part_at + size_t(p.splits) * p.batch * p.tokens * p.kv_heads * 2 * (p.dim <= 64 ? 64 : 128) * sizeof(float);
  if (!workspace) {
    *workspace_bytes = S.ws;
    return ZR_OK;
  }
  if (S.empty || (!grad_q && !grad_k && !grad_v)) return ZR_OK;
  if (!S.q.ptr || !S.k.ptr || !S.v.ptr || !S.go.ptr || !S.o.ptr || !lse) return ZR_ERR_NULL;
  if (*workspace_bytes < S.ws || reinterpret_cast<uintptr_t>(workspace) % 16) return ZR_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(low) % S.es || reinterpret_cast<uintptr_t>(lse) % 4) return ZR_ERR_LAYOUT;
  const Span in[] = {span_of(S.q.ptr, S.q.extent, S.es),   span_of(S.k.ptr, S.k.extent, S.es),
                     span_of(S.v.ptr, S.v.extent, S.es),   span_of(S.go.ptr, S.go.extent, S.es),
                     span_of(S.o.ptr, S.o.extent, S.es),   span_of(low, S.q.numel, S.es),
                     span_of(lse, S.q.numel / p.dim, 4),   span_of(offsets, int64_t(sequences) + 1, 4)};
  const Span outs[] = {span_of(grad_q, S.gq.extent, S.es), span_of(grad_k, S.gk.extent, S.es),
                       span_of(grad_v, S.gv.extent, S.es), span_of(workspace, int64_t(S.ws), 1)};
  // The gradients may be views that lie between one another, as those of one
  // projection's rows do: then their spans meet and their elements do not.
  const TDesc* grads[] = {&S.gq, &S.gk, &S.gv};
  for (int i = 0; i < 4; ++i)
    for (const Span& x : in)
      if (overlaps(outs[i], x)) return ZR_ERR_LAYOUT;
  for (int i = 0; i < 3; ++i) {
    if (overlaps(outs[i], outs[3])) return ZR_ERR_LAYOUT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j]) && !interleaved(*grads[i], *grads[j], S.es)) return ZR_ERR_LAYOUT;
  }
  p.go = view_of(S.go);
  p.o = view_of(S.o);
  p.gq = view_of(S.gq);
  p.gk = view_of(S.gk);
  p.gv = view_of(S.gv);
  p.low = const_cast<void*>(low);
  p.lse = const_cast<float*>(lse);
  p.lse2 = static_cast<float*>(workspace);
  p.delta = p.lse2 + rows;
  p.want = (grad_q ? 1u : 0u) | (grad_k ? 2u : 0u) | (grad_v ? 4u : 0u);
  p.vec = wide(S.q, S.es) && wide(S.k, S.es) && wide(S.v, S.es) && wide(S.go, S.es);
  p.o_wide = wide(S.o, S.es) && wide(S.go, S.es) && reinterpret_cast<uintptr_t>(low) % 16 == 0;
  p.g_wide = (wide(S.gq, S.es) ? 1u : 0u) | (wide(S.gk, S.es) ? 2u : 0u) | (wide(S.gv, S.es) ? 4u : 0u);
  if (tc) set_tiles(&p, 128);
  p.part = p.splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_at) : nullptr;
  trace("zr_attention_bwd", [&] { return plan_json(S, kernel_name(tc, copy, S.es)); });
  for (const void* x : {p.q.p, p.k.p, p.v.p, p.go.p, p.o.p, static_cast<const void*>(low),
                        static_cast<const void*>(lse), static_cast<const void*>(offsets),
                        static_cast<const void*>(grad_q), static_cast<const void*>(grad_k),
                        static_cast<const void*>(grad_v), static_cast<const void*>(workspace)})
    if (x && (rc = check_device_ptr(x))) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_attn_rows(S.es, p, st);
  if (e != cudaSuccess) return ZR_ERR_CUDA;
  if (!tc) return cuda_status(launch_attn_any_bwd(S.es, p, st));
  AttnMaps maps;
  e = operands(S, copy, copies, 4, workspace, &maps, st);
  if (e != cudaSuccess) return ZR_ERR_CUDA;
  return cuda_status(S.es == 4 ? launch_attn_f32_bwd(p, maps, st) : launch_attn_bwd(p, maps, st));
}

}  // namespace
}  // namespace zr

extern "C" {

int zr_attention_fwd(zr_dtype dtype, zr_tensor q, zr_tensor k, zr_tensor v, float scale,
                     const int32_t* offsets, int32_t sequences, void* out, const int64_t* out_strides,
                     void* low, float* lse, void* workspace, size_t* workspace_bytes, zr_stream_t stream) {
  return zr::fwd_impl(dtype, q, k, v, scale, offsets, sequences, out, out_strides, low, lse, workspace,
                      workspace_bytes, stream);
}

int zr_attention_bwd(zr_dtype dtype, zr_tensor grad_out, zr_tensor q, zr_tensor k, zr_tensor v,
                     zr_tensor out, const void* low, const float* lse, float scale,
                     const int32_t* offsets, int32_t sequences, void* grad_q,
                     const int64_t* grad_q_strides, void* grad_k, const int64_t* grad_k_strides,
                     void* grad_v, const int64_t* grad_v_strides, void* workspace,
                     size_t* workspace_bytes, zr_stream_t stream) {
  return zr::bwd_impl(dtype, grad_out, q, k, v, out, low, lse, scale, offsets, sequences, grad_q, grad_q_strides,
                      grad_k, grad_k_strides, grad_v, grad_v_strides, workspace, workspace_bytes, stream);
}

}  // extern "C"
