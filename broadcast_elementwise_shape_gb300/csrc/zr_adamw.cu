// zr_adamw.cu — AdamW over many tensors at once: kernels, plan and C entry
// points.
//
// Bound by HBM: per element 12 bytes of parameter and states read and 12
// written with binary32 states, 6 and 6 with 8-bit ones, the gradient and the
// bfloat16 copy besides.  So the tensors are cut into runs of 2048 elements, a
// CTA takes one, and the list of tensors goes to the kernel by value: one
// launch for some hundred tensors, nothing to copy to the device first.  124 M
// parameters: 522 us with binary32 states (7.1 TB/s), 418 with 8-bit ones (4.7: there
// the instructions bind, about 80 per element, a fifth of them the generator's;
// 516 us with three CTAs per SM and exact roots and quotients).
//
// 8-bit states.  A block's values, divided by its power of two, are multiplied
// by another power of two that puts the smallest normal code at the smallest
// normal binary32 number: exponent and mantissa of the code are then bits 20 and
// up of the binary32 pattern, subnormal codes included, and rounding up with
// the probability of what is cut off is the addition of a random number below
// 2^20 to the pattern.  Decoding is a shift and two exact multiplications.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "zr_checks.h"
#include "zr_kernels.cuh"
#include "zr_launch.h"
#include "zr_philox.cuh"

namespace zr {

constexpr uint32_t kAdamRun = kThreads * 8;  // elements of a CTA: a block of 256 per warp
constexpr int kAdamFew = 40, kAdamMany = 400;

struct AdamTensor {
  float* param;
  __nv_bfloat16* copy;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  uint32_t index;            // in the call
  float decay;               // lr * weight_decay; with a device lr weight_decay
};

// N tensors of one launch (kernel parameters are limited to 32,764 bytes; few
// tensors take a shorter list, of which each launch copies less).
template <int N>
struct AdamPlan {
  AdamTensor t[N];
  uint32_t first[N];         // first CTA of each
  uint32_t count;
  float b1, c1, b2, c2, eps; // c = 1 - b
  float rate;                // lr / (1 - beta1^t)
  float root;                // (1 - beta2^t)^-1/2
  float lr, log_b1, log_b2;  // with device values
  int64_t step;
  const int64_t* device_step;
  const float* device_lr;
  const float* device_scale;
  uint32_t key[20];
};
static_assert(sizeof(AdamPlan<kAdamMany>) < 32764, "kernel parameters");

namespace {

constexpr float kUnM = 0x1p113f, kUnV = 0x1p97f;  // code pattern -> value / scale

struct AdamFactors {
  float rate, root, decay, grad;
  int64_t step;
};

template <int N>
__device__ __forceinline__ AdamFactors adam_factors(const AdamPlan<N>& p, float decay) {
  AdamFactors f{p.rate, p.root, decay, 1.f, p.step};
  if (p.device_scale) f.grad = *p.device_scale;
  if (p.device_step || p.device_lr) {
    if (p.device_step) f.step += *p.device_step;
    const float lr = p.device_lr ? *p.device_lr : p.lr;
    const float t = float(f.step);
    f.rate = lr / -expm1f(t * p.log_b1);
    f.root = 1.f / sqrtf(-expm1f(t * p.log_b2));
    if (p.device_lr) f.decay = lr * decay;
  }
  return f;
}

template <int N>
__device__ __forceinline__ uint32_t adam_find(const AdamPlan<N>& p) {
  uint32_t lo = 0, hi = p.count;  // first[lo] <= blockIdx.x < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (p.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The root and the quotient are the hardware's approximate ones, within 2^-22: of
// the update, which is small beside the parameter, 2^-22 is far below the
// parameter's own rounding, and the exact forms take a quarter of the 8-bit
// step's instructions, which bound it.  (The states, whose codes depend on every bit,
// use neither.)
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void adam_one(float& param, float& m, float& v, float g, const AdamFactors& f,
                                         float b1, float c1, float b2, float c2, float eps) {
  g = __fmul_rn(g, f.grad);
  m = __fadd_rn(__fmul_rn(b1, m), __fmul_rn(c1, g));
  v = __fadd_rn(__fmul_rn(b2, v), __fmul_rn(c2, __fmul_rn(g, g)));
  const float d = __fadd_rn(__fmul_rn(sqrt_approx(v), f.root), eps);
  param = __fsub_rn(param, __fadd_rn(__fmul_rn(f.decay, param), __fmul_rn(f.rate, __fmul_rn(m, rcp_approx(d)))));
}

// The scale of a block whose largest magnitude has the pattern `top`, and its
// inverse; NaN where the block has no finite scale.
__device__ __forceinline__ void adam_scale(uint32_t top, float& scale, float& inverse) {
  const int e = max(int(top >> 23) - 127, -90);
  const bool bad = e >= 127;
  scale = bad ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(uint32_t(127 + e) << 23);
  inverse = bad ? 0.f : __uint_as_float(uint32_t(127 - e) << 23);
}
__device__ __forceinline__ uint32_t adam_code(float x, float inverse, float un, uint32_t cut) {
  return (__float_as_uint(__fmul_rn(__fmul_rn(fabsf(x), inverse), 1.f / un)) + cut) >> 20;
}
__device__ __forceinline__ float adam_m(uint32_t code, float scale) {
  const float x = __fmul_rn(__fmul_rn(__uint_as_float((code & 127u) << 20), kUnM), scale);
  return code & 128u ? -x : x;
}
__device__ __forceinline__ float adam_v(uint32_t code, float scale) {
  return __fmul_rn(__fmul_rn(__uint_as_float(code << 20), kUnV), scale);
}

// A warp's 256 elements, 8 per lane.  W = 4: in two groups of four neighbours
// at `lane * 4` and 128 behind, read as vectors; W = 1 (pointers at odd
// addresses): 32 apart.
template <int W>
__device__ __forceinline__ uint32_t adam_place(int k, uint32_t lane) {
  return W == 4 ? lane * 4 + (k / 4) * 128 + k % 4 : lane + k * 32;
}

template <typename T, int W>
__device__ __forceinline__ void adam_load(const T* from, uint32_t n, uint32_t lane, T* to) {
  if constexpr (W == 4) {
    if (n >= 256) {
      struct alignas(sizeof(T) * 4) Vec { T e[4]; };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Vec x = *reinterpret_cast<const Vec*>(from + lane * 4 + h * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) to[4 * h + k] = x.e[k];
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t e = adam_place<W>(k, lane);
    to[k] = e < n ? from[e] : T();
  }
}
template <typename T, int W>
__device__ __forceinline__ void adam_store(T* to, uint32_t n, uint32_t lane, const T* from) {
  if constexpr (W == 4) {
    if (n >= 256) {
      struct alignas(sizeof(T) * 4) Vec { T e[4]; };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Vec x;
#pragma unroll
        for (int k = 0; k < 4; ++k) x.e[k] = from[4 * h + k];
        *reinterpret_cast<Vec*>(to + lane * 4 + h * 128) = x;
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t e = adam_place<W>(k, lane);
    if (e < n) to[e] = from[k];
  }
}

template <typename G>
__device__ __forceinline__ float adam_grad(G g) {
  if constexpr (sizeof(G) == 4) return g;
  else return __uint_as_float(uint32_t(g) << 16);
}

template <typename G, int BITS, int W, int N>
__device__ __forceinline__ void adam_block(const AdamPlan<N>& p, const AdamTensor& t, int64_t at,
                                           uint32_t n, uint32_t lane, uint32_t* words) {
  float param[8], m[8], v[8];
  G g[8];
  uint8_t mc[8], vc[8];
  float ms = 0.f, vs = 0.f;
  adam_load<float, W>(t.param + at, n, lane, param);
  adam_load<G, W>(static_cast<const G*>(t.grad) + at, n, lane, g);
  if constexpr (BITS == 8) {
    adam_load<uint8_t, W>(static_cast<const uint8_t*>(t.m) + at, n, lane, mc);
    adam_load<uint8_t, W>(static_cast<const uint8_t*>(t.v) + at, n, lane, vc);
    ms = t.m_scale[at / ZR_ADAMW_BLOCK];
    vs = t.v_scale[at / ZR_ADAMW_BLOCK];
  } else {
    adam_load<float, W>(static_cast<const float*>(t.m) + at, n, lane, m);
    adam_load<float, W>(static_cast<const float*>(t.v) + at, n, lane, v);
  }
  const AdamFactors f = adam_factors(p, t.decay);
  uint32_t w[8];
  if constexpr (BITS == 8) {
    // Two counters per lane, eight words, as many as it has elements.  Their
    // elements are neighbours; with W = 1 the words change lanes through shared
    // memory.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t c = uint64_t(at) / 4 + lane + h * 32;
      philox(uint32_t(c), t.index, uint32_t(f.step), uint32_t(uint64_t(f.step) >> 32), p.key, w + 4 * h);
      if (W == 1)
        *reinterpret_cast<uint4*>(words + lane * 4 + h * 128) =
            make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    }
    if (W == 1) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = words[lane + k * 32];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = adam_m(mc[k], ms);
      v[k] = adam_v(vc[k], vs);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    adam_one(param[k], m[k], v[k], adam_grad(g[k]), f, p.b1, p.c1, p.b2, p.c2, p.eps);
  adam_store<float, W>(t.param + at, n, lane, param);
  if (t.copy) {
    uint16_t c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = __bfloat16_as_ushort(__float2bfloat16_rn(param[k]));
    adam_store<uint16_t, W>(reinterpret_cast<uint16_t*>(t.copy) + at, n, lane, c);
  }
  if constexpr (BITS == 8) {
    uint32_t tm = 0, tv = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (adam_place<W>(k, lane) < n) {  // elements behind the end are no part of the block
        tm = max(tm, __float_as_uint(fabsf(m[k])));
        tv = max(tv, __float_as_uint(fabsf(v[k])));
      }
    }
    tm = __reduce_max_sync(0xFFFFFFFFu, tm);
    tv = __reduce_max_sync(0xFFFFFFFFu, tv);
    float mi, vi;
    adam_scale(tm, ms, mi);
    adam_scale(tv, vs, vi);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      mc[k] = uint8_t(adam_code(m[k], mi, kUnM, (w[k] & 0xFFFFu) << 4 | 8u) | (__float_as_uint(m[k]) >> 31 << 7));
      vc[k] = uint8_t(adam_code(v[k], vi, kUnV, (w[k] >> 16) << 4 | 8u));
    }
    adam_store<uint8_t, W>(static_cast<uint8_t*>(t.m) + at, n, lane, mc);
    adam_store<uint8_t, W>(static_cast<uint8_t*>(t.v) + at, n, lane, vc);
    if (lane == 0) {
      t.m_scale[at / ZR_ADAMW_BLOCK] = ms;
      t.v_scale[at / ZR_ADAMW_BLOCK] = vs;
    }
  } else {
    adam_store<float, W>(static_cast<float*>(t.m) + at, n, lane, m);
    adam_store<float, W>(static_cast<float*>(t.v) + at, n, lane, v);
  }
}

template <typename G, int BITS, int N>
__global__ void __launch_bounds__(kThreads, 4) k_adamw(const __grid_constant__ AdamPlan<N> p) {
  __shared__ __align__(16) uint32_t s_words[BITS == 8 ? kAdamRun : 4];
  pdl_trigger();
  const uint32_t i = adam_find(p);
  const AdamTensor& t = p.t[i];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t at = int64_t(blockIdx.x - p.first[i]) * kAdamRun + warp * 256;
  pdl_wait();
  if (at >= t.n) return;
  const uint32_t n = t.n - at < 256 ? uint32_t(t.n - at) : 256;
  uint32_t* words = s_words + (BITS == 8 ? warp * 256 : 0);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.copy) * 2 |
                         reinterpret_cast<uintptr_t>(t.grad) * (4 / sizeof(G)) |
                         (reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) * (32 / BITS);
  if (bits % 16 == 0) adam_block<G, BITS, 4>(p, t, at, n, lane, words);
  else adam_block<G, BITS, 1>(p, t, at, n, lane, words);
}

// The values of 8-bit states (param: m's values, copy: v's; either may be null).
template <int N>
__global__ void __launch_bounds__(kThreads) k_adamw_state(const __grid_constant__ AdamPlan<N> p) {
  pdl_trigger();
  const uint32_t i = adam_find(p);
  const AdamTensor& t = p.t[i];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t at = int64_t(blockIdx.x - p.first[i]) * kAdamRun + warp * 256;
  pdl_wait();
  if (at >= t.n) return;
  const uint32_t n = t.n - at < 256 ? uint32_t(t.n - at) : 256;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint16_t* out = which ? reinterpret_cast<uint16_t*>(t.copy) : reinterpret_cast<uint16_t*>(t.param);
    if (!out) continue;
    const uint8_t* in = static_cast<const uint8_t*>(which ? t.v : t.m) + at;
    const float s = (which ? t.v_scale : t.m_scale)[at / ZR_ADAMW_BLOCK];
    const auto value = [&](uint32_t c) {
      return uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(which ? adam_v(c, s) : adam_m(c, s))));
    };
    if (n == 256 && (reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(in) * 2) % 16 == 0) {
      const uint2 c = *reinterpret_cast<const uint2*>(in + lane * 8);
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t two = (k < 2 ? c.x : c.y) >> (k % 2 * 16);
        o[k] = value(two & 255) | value(two >> 8 & 255) << 16;
      }
      *reinterpret_cast<uint4*>(out + at + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      uint8_t c[8];
      uint16_t o[8];
      adam_load<uint8_t, 1>(in, n, lane, c);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = uint16_t(value(c[k]));
      adam_store<uint16_t, 1>(out + at, n, lane, o);
    }
  }
}

// One buffer of the call.
struct AdamSpan {
  uintptr_t lo, hi;
  bool written;
};

// No written buffer may share a byte with another; every buffer is memory that
// the device addresses.  Sorted, both take one walk; buffers out of one
// allocation are looked up once (a lookup costs some hundred ns, a call has up
// to seven buffers a tensor).  The buffers of one kind mostly ascend already, as
// views of one large buffer do, so the sort merges the runs it finds.
int check_spans(std::vector<AdamSpan>& s) {
  const auto before = [](const AdamSpan& x, const AdamSpan& y) { return x.lo < y.lo; };
  std::vector<size_t> run{0};
  for (size_t i = 1; i < s.size(); ++i)
    if (before(s[i], s[i - 1])) run.push_back(i);
  run.push_back(s.size());
  std::vector<AdamSpan> to(s.size());
  while (run.size() > 2) {
    std::vector<size_t> next;
    for (size_t r = 0; r + 1 < run.size(); r += 2) {
      const auto from = [&](size_t k) { return s.begin() + std::ptrdiff_t(run[std::min(r + k, run.size() - 1)]); };
      std::merge(from(0), from(1), from(1), from(2), to.begin() + std::ptrdiff_t(run[r]), before);
      next.push_back(run[r]);
    }
    next.push_back(s.size());
    run.swap(next);
    s.swap(to);
  }
  uintptr_t any = 0, written = 0;
  for (const AdamSpan& x : s) {
    if (x.lo < written || (x.written && x.lo < any)) return ZR_ERR_LAYOUT;
    any = std::max(any, x.hi);
    if (x.written) written = std::max(written, x.hi);
  }
  return ZR_OK;
}
int check_devices(const std::vector<AdamSpan>& s) {
  uintptr_t known = 0;  // up to here the last buffer's allocation reaches
  using RangeFn = CUresult (*)(CUdeviceptr*, size_t*, CUdeviceptr);
  static const RangeFn range = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<RangeFn>(f);
  }();
  for (const AdamSpan& x : s) {
    if (x.lo < known) continue;
    const int rc = check_device_ptr(reinterpret_cast<const void*>(x.lo));
    if (rc) return rc;
    CUdeviceptr base = 0;
    size_t bytes = 0;
    known = range && range(&base, &bytes, CUdeviceptr(x.lo)) == CUDA_SUCCESS ? uintptr_t(base) + bytes : 0;
  }
  return ZR_OK;
}

void add_span(std::vector<AdamSpan>& s, const void* p, int64_t n, int es, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (lo) s.push_back({lo, lo + uintptr_t(n) * uintptr_t(es), written});
}
int64_t scales_of(int64_t n) { return (n + ZR_ADAMW_BLOCK - 1) / ZR_ADAMW_BLOCK; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Launches `run` for the tensors' elements, kAdamMany tensors at a time.
template <typename Few, typename Many>
cudaError_t adam_launch(const std::vector<AdamTensor>& list, const AdamPlan<1>& with, Few few, Many many) {
  const auto group = [&](auto& p, size_t at, size_t n, auto& run) {
    p.b1 = with.b1; p.c1 = with.c1; p.b2 = with.b2; p.c2 = with.c2; p.eps = with.eps;
    p.rate = with.rate; p.root = with.root;
    p.lr = with.lr; p.log_b1 = with.log_b1; p.log_b2 = with.log_b2;
    p.step = with.step;
    p.device_step = with.device_step; p.device_lr = with.device_lr; p.device_scale = with.device_scale;
    std::copy(with.key, with.key + 20, p.key);
    p.count = uint32_t(n);
    uint32_t cta = 0;
    for (size_t i = 0; i < n; ++i) {
      p.t[i] = list[at + i];
      p.first[i] = cta;
      cta += uint32_t((list[at + i].n + kAdamRun - 1) / kAdamRun);
    }
    return run(p, cta);
  };
  for (size_t at = 0; at < list.size();) {
    // A grid has at most 2^31 - 1 CTAs.
    size_t n = 0;
    for (uint64_t cta = 0; at + n < list.size() && n < size_t(kAdamMany); ++n) {
      cta += uint64_t(list[at + n].n + kAdamRun - 1) / kAdamRun;
      if (n && cta >= (uint64_t(1) << 31)) break;
    }
    cudaError_t e;
    if (n <= size_t(kAdamFew)) {
      AdamPlan<kAdamFew> p{};
      e = group(p, at, n, few);
    } else {
      AdamPlan<kAdamMany> p{};
      e = group(p, at, n, many);
    }
    if (e != cudaSuccess) return e;
    at += n;
  }
  return cudaSuccess;
}

constexpr int64_t kMostElements = int64_t(1) << 40;  // its CTAs fit a grid, its bytes 64 bits

int step_impl(zr_dtype grad_type, int32_t state_bits, int32_t count, const zr_adamw_tensor* tensors,
              const zr_adamw* how, zr_stream_t stream) {
  if (!how || count < 0 || (count > 0 && !tensors)) return count < 0 ? ZR_ERR_SIZE : ZR_ERR_NULL;
  if (grad_type != ZR_F32 && grad_type != ZR_BF16) return ZR_ERR_DTYPE;
  if (state_bits != 8 && state_bits != 32) return ZR_ERR_DTYPE;
  const auto beta = [](double b) { return b >= 0 && b < 1 && float(b) < 1.f; };
  if (!std::isfinite(how->lr) || !beta(how->beta1) || !beta(how->beta2) || !(how->eps >= 0) ||
      !std::isfinite(how->eps) || how->step < 1)
    return ZR_ERR_VALUE;
  const int gs = grad_type == ZR_BF16 ? 2 : 4;
  std::vector<AdamTensor> list;
  std::vector<AdamSpan> spans;
  list.reserve(size_t(count));
  spans.reserve(size_t(count) * 7 + 3);
  const int ss = state_bits / 8;
  for (int32_t i = 0; i < count; ++i) {
    const zr_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (state_bits == 8 ? int64_t(1) << 34 : kMostElements)) return ZR_ERR_SIZE;
    if (!std::isfinite(t.weight_decay)) return ZR_ERR_VALUE;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale))) return ZR_ERR_NULL;
    if (!aligned(t.param, 4) || !aligned(t.grad, gs) || !aligned(t.m, ss) || !aligned(t.v, ss) || !aligned(t.copy, 2) ||
        (state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
      return ZR_ERR_LAYOUT;
    const float decay = how->device_lr ? t.weight_decay : float(how->lr * double(t.weight_decay));
    list.push_back({t.param, static_cast<__nv_bfloat16*>(t.copy), t.grad, t.m, t.v, t.m_scale, t.v_scale, t.n,
                    uint32_t(i), decay});
  }
  for (const AdamTensor& t : list) add_span(spans, t.param, t.n, 4, true);
  for (const AdamTensor& t : list) add_span(spans, t.grad, t.n, gs, false);
  for (const AdamTensor& t : list) add_span(spans, t.m, t.n, ss, true);
  for (const AdamTensor& t : list) add_span(spans, t.v, t.n, ss, true);
  for (const AdamTensor& t : list) add_span(spans, t.copy, t.n, 2, true);
  if (state_bits == 8) {
    for (const AdamTensor& t : list) add_span(spans, t.m_scale, scales_of(t.n), 4, true);
    for (const AdamTensor& t : list) add_span(spans, t.v_scale, scales_of(t.n), 4, true);
  }
  if (list.empty()) return ZR_OK;
  if (how->device_step) add_span(spans, how->device_step, 1, 8, false);
  if (how->device_lr) add_span(spans, how->device_lr, 1, 4, false);
  if (how->device_grad_scale) add_span(spans, how->device_grad_scale, 1, 4, false);
  if (!aligned(how->device_step, 8) || !aligned(how->device_lr, 4) || !aligned(how->device_grad_scale, 4))
    return ZR_ERR_LAYOUT;
  int rc = check_spans(spans);
  if (rc) return rc;
  trace("zr_adamw_step", [&] {
    return std::string("{\"kernel\":\"adamw\",\"tensors\":") + std::to_string(list.size()) +
           ",\"bits\":" + std::to_string(state_bits) + "}";
  });
  if ((rc = check_devices(spans))) return rc;
  AdamPlan<1> w{};
  w.b1 = float(how->beta1);
  w.c1 = float(1.0 - how->beta1);
  w.b2 = float(how->beta2);
  w.c2 = float(1.0 - how->beta2);
  w.eps = float(how->eps);
  const double t = double(how->step);
  w.rate = float(how->lr / (1.0 - std::pow(how->beta1, t)));
  w.root = float(1.0 / std::sqrt(1.0 - std::pow(how->beta2, t)));
  w.lr = float(how->lr);
  w.log_b1 = float(std::log(how->beta1));
  w.log_b2 = float(std::log(how->beta2));
  w.step = how->step;
  w.device_step = how->device_step;
  w.device_lr = how->device_lr;
  w.device_scale = how->device_grad_scale;
  philox_keys(how->seed, w.key);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const auto run = [&](const auto& p, uint32_t cta) {
    constexpr int N = int(sizeof(p.first) / sizeof(uint32_t));
    const auto k = state_bits == 8 ? (gs == 2 ? k_adamw<uint16_t, 8, N> : k_adamw<float, 8, N>)
                                   : (gs == 2 ? k_adamw<uint16_t, 32, N> : k_adamw<float, 32, N>);
    return launch_k(k, cta, kThreads, 0, st, p);
  };
  return cuda_status(adam_launch(list, w, run, run));
}

int state_impl(int32_t count, const zr_adamw_tensor* tensors, void* const* m_out, void* const* v_out,
               zr_stream_t stream) {
  if (count < 0) return ZR_ERR_SIZE;
  if (count > 0 && !tensors) return ZR_ERR_NULL;
  std::vector<AdamTensor> list;
  std::vector<AdamSpan> spans;
  list.reserve(size_t(count));
  spans.reserve(size_t(count) * 6);
  for (int32_t i = 0; i < count; ++i) {
    const zr_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= int64_t(1) << 34) return ZR_ERR_SIZE;
    void* om = m_out ? m_out[i] : nullptr;
    void* ov = v_out ? v_out[i] : nullptr;
    if (t.n == 0 || (!om && !ov)) continue;
    if ((om && (!t.m || !t.m_scale)) || (ov && (!t.v || !t.v_scale))) return ZR_ERR_NULL;
    if (!aligned(om, 2) || !aligned(ov, 2) || (om && !aligned(t.m_scale, 4)) || (ov && !aligned(t.v_scale, 4)))
      return ZR_ERR_LAYOUT;
    list.push_back({static_cast<float*>(om), static_cast<__nv_bfloat16*>(ov), nullptr, t.m, t.v, t.m_scale,
                    t.v_scale, t.n, uint32_t(i), 0.f});
  }
  if (list.empty()) return ZR_OK;
  for (int which = 0; which < 2; ++which) {
    const auto out = [&](const AdamTensor& t) { return which ? static_cast<void*>(t.copy) : static_cast<void*>(t.param); };
    for (const AdamTensor& t : list) add_span(spans, out(t), t.n, 2, true);
    for (const AdamTensor& t : list)
      if (out(t)) add_span(spans, which ? t.v : t.m, t.n, 1, false);
    for (const AdamTensor& t : list)
      if (out(t)) add_span(spans, which ? t.v_scale : t.m_scale, scales_of(t.n), 4, false);
  }
  int rc = check_spans(spans);
  if (rc) return rc;
  trace("zr_adamw_state", [&] {
    return std::string("{\"kernel\":\"adamw_state\",\"tensors\":") + std::to_string(list.size()) + "}";
  });
  if ((rc = check_devices(spans))) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const auto run = [&](const auto& p, uint32_t cta) {
    constexpr int N = int(sizeof(p.first) / sizeof(uint32_t));
    return launch_k(k_adamw_state<N>, cta, kThreads, 0, st, p);
  };
  return cuda_status(adam_launch(list, AdamPlan<1>{}, run, run));
}

}  // namespace
}  // namespace zr

extern "C" {

int zr_adamw_step(zr_dtype grad_type, int32_t state_bits, int32_t count,
                  const zr_adamw_tensor* tensors, const zr_adamw* how, zr_stream_t stream) {
  try {
    return zr::step_impl(grad_type, state_bits, count, tensors, how, stream);
  } catch (...) {  // no memory for the lists
    return ZR_ERR_MEMORY;
  }
}

int zr_adamw_state(int32_t count, const zr_adamw_tensor* tensors, void* const* m_out,
                   void* const* v_out, zr_stream_t stream) {
  try {
    return zr::state_impl(count, tensors, m_out, v_out, stream);
  } catch (...) {
    return ZR_ERR_MEMORY;
  }
}

}  // extern "C"
