// zr_dropout.cu — dropout with a residual: kernels, plan and C entry points.
//
// out[i] = residual[i] + (keep(i) ? x[i] * scale : 0), scale = 1 / (1 - p);
// the backward is the same without a residual, on the gradient.  keep(i) is
// computed where it is needed and never stored: element i (row-major over
// the shape, whatever the strides) takes word i mod 4 of the counter-based
// generator Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror and
// D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at
// counter offset + i div 4 under the seed as key, and is kept when the word
// is at least round(p * 2^32).  So forward and backward agree without any
// memory between them, on every layout and launch shape.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "zr_checks.h"
#include "zr_kernels.cuh"
#include "zr_launch.h"
#include "zr_philox.cuh"

namespace zr {

// Slots: 0 x (or the gradient), 1 residual, 3 out.
struct DropPlan {
  const void* x;
  const void* residual;      // or null
  void* out;
  const uint64_t* device_offset;  // added to offset, or null
  uint64_t offset;
  uint32_t key[20];          // the seed's ten round keys
  Decomp rows;
  int64_t inner_stride[kMaxOperands];
  uint64_t numel;
  uint64_t nitems;           // vector plans: vectors; else ceil(numel / 4)
  uint32_t ncol, nvcol;
  uint32_t one_row;          // every operand is one dense run (no rows, ncol unused)
  uint32_t last_drop;        // keep = keep_all or word > last_drop
  uint32_t keep_all;
  float scale;
};

namespace {

__device__ __forceinline__ void philox(uint64_t counter, const uint32_t* key, uint32_t* w) {
  zr::philox(uint32_t(counter), uint32_t(counter >> 32), 0, 0, key, w);
}

template <typename E, bool RES>
__device__ __forceinline__ void dropout_one(const DropPlan& p, uint32_t word, int64_t x_off,
                                            int64_t r_off, int64_t o_off) {
  const float x = ld1(static_cast<const E*>(p.x) + x_off, false);
  const bool keep = p.keep_all || word > p.last_drop;
  float y = keep ? __fmul_rn(x, p.scale) : 0.f;
  if (RES) y = __fadd_rn(ld1(static_cast<const E*>(p.residual) + r_off, false), y);
  st1(static_cast<E*>(p.out) + o_off, y);
}

// 16-byte vectors: VEC consecutive elements of one row, VEC / 4 counters.  Must
// read x and the residual and write out; what bounds it is at drop_unroll.
template <typename E, int VEC, bool RES, int U>
__global__ void __launch_bounds__(kThreads) k_dropout_vec(const __grid_constant__ DropPlan p) {
  pdl_trigger();
  const uint64_t first = uint64_t(blockIdx.x) * (kThreads * U) + threadIdx.x;
  pdl_wait();
  const uint64_t base = p.offset + (p.device_offset ? *p.device_offset : 0);
  uint4 xv[U], rv[U];
  int64_t oo[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t i = first + uint64_t(u) * kThreads;
    if (i >= p.nitems) continue;
    int64_t off[kMaxOperands];
    if (p.one_row) {
      off[0] = off[1] = off[kSlotOut] = int64_t(i) * VEC;
    } else {
      const uint32_t row = uint32_t(i / p.nvcol);
      const int64_t c = int64_t(i - uint64_t(row) * p.nvcol) * VEC;
      decomp_offsets(p.rows, row, off);
      off[0] += c; off[1] += c; off[kSlotOut] += c;
    }
    oo[u] = off[kSlotOut];
    if ((i + 1) * VEC > p.numel) continue;  // the run's ragged end, below
    xv[u] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.x) + off[0]);
    if (RES) rv[u] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.residual) + off[1]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t i = first + uint64_t(u) * kThreads;
    if (i >= p.nitems) continue;
    if ((i + 1) * VEC > p.numel) {
      for (uint64_t e = i * VEC; e < p.numel; ++e) {
        uint32_t w[4];
        philox(base + e / 4, p.key, w);
        const uint32_t word = e % 4 == 0 ? w[0] : e % 4 == 1 ? w[1] : e % 4 == 2 ? w[2] : w[3];
        dropout_one<E, RES>(p, word, int64_t(e), int64_t(e), int64_t(e));
      }
      continue;
    }
    const uint32_t xw[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
    uint32_t rw[4] = {0, 0, 0, 0}, ow[4];
    if (RES) { rw[0] = rv[u].x; rw[1] = rv[u].y; rw[2] = rv[u].z; rw[3] = rv[u].w; }
    float o[VEC];
#pragma unroll
    for (int b = 0; b < VEC / 4; ++b) {
      uint32_t w[4];
      philox(base + i * (VEC / 4) + b, p.key, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * b + j;
        float x, r;
        if constexpr (sizeof(E) == 4) {
          x = __uint_as_float(xw[e]);
          r = __uint_as_float(rw[e]);
        } else {
          x = __uint_as_float(e & 1 ? xw[e / 2] & 0xFFFF0000u : xw[e / 2] << 16);
          r = __uint_as_float(e & 1 ? rw[e / 2] & 0xFFFF0000u : rw[e / 2] << 16);
        }
        const bool keep = p.keep_all || w[j] > p.last_drop;
        const float y = keep ? __fmul_rn(x, p.scale) : 0.f;
        o[e] = RES ? __fadd_rn(r, y) : y;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(E) == 4) {
        ow[k] = __float_as_uint(o[k]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
        ow[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<E*>(p.out) + oo[u]) =
        make_uint4(ow[0], ow[1], ow[2], ow[3]);
  }
}

// Any strides: a thread takes the four elements of one counter.
template <typename E, bool RES>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const __grid_constant__ DropPlan p) {
  pdl_trigger();
  const uint64_t i = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
  pdl_wait();
  if (i >= p.nitems) return;
  const uint64_t base = p.offset + (p.device_offset ? *p.device_offset : 0);
  uint32_t w[4];
  philox(base + i, p.key, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t e = 4 * i + j;
    if (e >= p.numel) return;
    int64_t off[kMaxOperands];
    if (p.one_row) {
      off[0] = off[1] = off[kSlotOut] = int64_t(e);
    } else {
      const uint32_t row = uint32_t(e / p.ncol);
      const int64_t c = int64_t(e - uint64_t(row) * p.ncol);
      decomp_offsets(p.rows, row, off);
#pragma unroll
      for (int k = 0; k < kMaxOperands; ++k) off[k] += c * p.inner_stride[k];
    }
    dropout_one<E, RES>(p, w[j], off[0], off[1], off[kSlotOut]);
  }
}

// Vectors per thread, loaded before the first is used.  binary32 is bound by
// HBM (without a residual [65536, 1536] 120 us with 3 and 127 with 1, with one
// [16384, 768] 21.7 us with 2 and 22.8 with 4); bfloat16 by the generator's
// integer multiplications (25 M counters in 95 us), where more warps help
// ([16384, 768] with a residual 14.3 us with 2 and 16.1 with 4).
ZR_CX int drop_unroll(int es, bool residual) { return es == 4 && !residual ? 3 : 2; }

struct DropSet {
  int es = 4, vec = 1;
  bool empty = false;
  DropPlan p;
  TDesc x, r, out;
  uint64_t n_cta = 0;
};

template <typename E, int VEC>
cudaError_t launch(const DropSet& S, cudaStream_t s) {
  const DropPlan& p = S.p;
  const unsigned n = unsigned(S.n_cta);
  if (S.vec == 1)
    return p.residual ? launch_k(k_dropout_any<E, true>, n, kThreads, 0, s, p)
                      : launch_k(k_dropout_any<E, false>, n, kThreads, 0, s, p);
  constexpr int es = sizeof(E);
  return p.residual
             ? launch_k(k_dropout_vec<E, VEC, true, drop_unroll(es, true)>, n, kThreads, 0, s, p)
             : launch_k(k_dropout_vec<E, VEC, false, drop_unroll(es, false)>, n, kThreads, 0, s, p);
}

int plan_dropout(zr_dtype dtype, const zr_tensor& x, const zr_tensor* residual, double prob,
                 const zr_rng& rng, void* out, const int64_t* out_strides, DropSet* S) {
  if (dtype != ZR_F32 && dtype != ZR_BF16) return ZR_ERR_DTYPE;
  S->es = dtype == ZR_BF16 ? 2 : 4;
  DropPlan& p = S->p;
  p = DropPlan{};
  if (!(prob >= 0.0 && prob <= 1.0)) return ZR_ERR_VALUE;
  int rc = read_tensor(x, &S->x);
  if (rc) return rc;
  const int n = S->x.nd;
  S->r = TDesc{};
  const bool res = residual && residual->data;
  if (res) {
    if ((rc = read_tensor(*residual, &S->r))) return rc;
    if (S->r.nd != n) return ZR_ERR_SHAPE;
    for (int d = 0; d < n; ++d)
      if (S->r.size[d] != S->x.size[d]) return ZR_ERR_SHAPE;
  }
  if ((rc = read_tensor(zr_tensor{out, n, S->x.size, out_strides}, &S->out))) return rc;
  if (S->x.numel == 0) {
    S->empty = true;
    return ZR_OK;
  }
  if (!S->x.ptr || !out) return ZR_ERR_NULL;
  if (!non_overlapping(S->out)) return ZR_ERR_LAYOUT;
  const Span so = span_of(out, S->out.extent, S->es);
  for (const TDesc* t : {&S->x, &S->r})
    if (overlaps(so, span_of(t->ptr, t->extent, S->es)) && !same_layout(*t, S->out))
      return ZR_ERR_LAYOUT;
  const uintptr_t dev_off = reinterpret_cast<uintptr_t>(rng.device_offset);
  if (dev_off % 8 != 0) return ZR_ERR_LAYOUT;
  if (overlaps(so, span_of(rng.device_offset, rng.device_offset ? 1 : 0, 8))) return ZR_ERR_LAYOUT;

  p.x = S->x.ptr;
  p.residual = res ? S->r.ptr : nullptr;
  p.out = out;
  p.device_offset = rng.device_offset;
  philox_keys(rng.seed, p.key);
  p.offset = rng.offset;
  p.numel = uint64_t(S->x.numel);
  const double thr = std::nearbyint(prob * 4294967296.0);
  p.keep_all = thr < 1.0;
  p.last_drop = p.keep_all ? 0u : uint32_t(uint64_t(thr) - 1);
  p.scale = prob < 1.0 ? float(1.0 / (1.0 - prob)) : 0.f;

  const int V = 16 / S->es;
  const void* ptr[kMaxOperands] = {p.x, p.residual, nullptr, out};
  const TDesc* desc[kMaxOperands] = {&S->x, &S->r, nullptr, &S->out};
  const uint32_t slots = 1u | (res ? 2u : 0u) | (1u << kSlotOut);
  bool wide = true, dense = true;
  int64_t cs[kMaxDims];
  contiguous_strides(n, S->x.size, cs);
  for (int k = 0; k < kMaxOperands; ++k) {
    if (!(slots & (1u << k))) continue;
    if (reinterpret_cast<uintptr_t>(ptr[k]) % 16 != 0) wide = false;
    for (int d = 0; d < n; ++d)
      if (S->x.size[d] != 1 && desc[k]->stride[d] != cs[d]) dense = false;
  }
  if (dense) {
    p.one_row = 1;
    p.nitems = (p.numel + V - 1) / V;
  } else {
    int64_t st[kProbSlots][kMaxDims] = {};
    for (int d = 0; d < n; ++d) {
      if (S->x.size[d] == 1) continue;
      for (int k = 0; k < kMaxOperands; ++k)
        if (slots & (1u << k)) st[k][d] = desc[k]->stride[d];
    }
    Prob P;
    // -1: the index stays row-major over the shape, as the generator counts.
    if ((rc = coalesce(n, S->x.size, st, slots, -1, &P))) return rc;
    const int in = P.n - 1;
    p.rows.n = in;
    uint64_t nrow = 1;
    for (int i = 0; i < in; ++i) {
      const int d = in - 1 - i;
      p.rows.div[i] = make_fastdiv(uint32_t(P.size[d]));
      for (int k = 0; k < kMaxOperands; ++k) p.rows.stride[k][i] = P.st[k][d];
      nrow *= uint64_t(P.size[d]);
      if (nrow >= (uint64_t(1) << 32)) return ZR_ERR_SIZE;
    }
    p.ncol = uint32_t(P.size[in]);
    if (p.ncol % uint32_t(V) != 0) wide = false;
    for (int k = 0; k < kMaxOperands; ++k) {
      p.inner_stride[k] = P.st[k][in];
      if (!(slots & (1u << k))) continue;
      if (p.inner_stride[k] != 1) wide = false;
      for (int i = 0; i < in; ++i)
        if (p.rows.stride[k][i] % V != 0) wide = false;
    }
    p.nvcol = p.ncol / uint32_t(V);
    p.nitems = nrow * p.nvcol;
  }
  S->vec = wide ? V : 1;
  if (!wide) p.nitems = (p.numel + 3) / 4;
  const uint64_t per = uint64_t(kThreads) * (wide ? drop_unroll(S->es, res) : 1);
  S->n_cta = (p.nitems + per - 1) / per;
  return S->n_cta < (uint64_t(1) << 31) ? ZR_OK : ZR_ERR_SIZE;
}

int run_dropout(const char* name, zr_dtype dtype, const zr_tensor& x, const zr_tensor* residual,
                double prob, const zr_rng& rng, void* out, const int64_t* out_strides,
                zr_stream_t stream) {
  DropSet S;
  int rc = plan_dropout(dtype, x, residual, prob, rng, out, out_strides, &S);
  if (rc || S.empty) return rc;
  trace(name, [&] {
    return std::string("{\"kernel\":\"dropout\",\"vec\":") + std::to_string(S.vec) +
           ",\"items\":" + std::to_string(S.p.nitems) + ",\"n_cta\":" + std::to_string(S.n_cta) + "}";
  });
  const void* need[4] = {S.p.x, S.p.residual, out, rng.device_offset};
  for (const void* q : need)
    if (q && (rc = check_device_ptr(q))) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(S.es == 2 ? launch<__nv_bfloat16, 8>(S, st) : launch<float, 4>(S, st));
}

}  // namespace
}  // namespace zr

extern "C" {

int zr_dropout_fwd(zr_dtype dtype, zr_tensor x, zr_tensor residual, double p, zr_rng rng, void* out,
                   const int64_t* out_strides, zr_stream_t stream) {
  return zr::run_dropout("zr_dropout_fwd", dtype, x, &residual, p, rng, out, out_strides, stream);
}

int zr_dropout_bwd(zr_dtype dtype, zr_tensor grad_out, double p, zr_rng rng, void* grad_x,
                   const int64_t* grad_x_strides, zr_stream_t stream) {
  return zr::run_dropout("zr_dropout_bwd", dtype, grad_out, nullptr, p, rng, grad_x, grad_x_strides,
                         stream);
}

}  // extern "C"
