// zr_packed.cpp — the packed-argument forms of the training operators
// (include/zr_packed.h): unpack and call the zr.h function.
#include "../../include/zr_packed.h"

#include <cstring>

namespace {

struct Reader {
  const int64_t* w;
  bool ok = true;

  double real() {
    double d;
    std::memcpy(&d, w++, sizeof d);
    return d;
  }
  int64_t i64() { return *w++; }
  template <typename T>
  T* ptr() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(*w++));
  }
  zr_tensor tensor() {
    zr_tensor t{};
    if (!ok) return t;
    t.data = ptr<void>();
    const int64_t nd = *w++;
    if (nd < 0 || nd > ZR_MAX_DIMS) {
      ok = false;
      return t;
    }
    t.ndim = int32_t(nd);
    t.sizes = w;
    t.strides = w + nd;
    w += 2 * nd;
    return t;
  }
};

// Runs call(workspace, &bytes); where the workspace given is too small, *need
// becomes the size it should have.
template <typename F>
int with_need(void* ws, int64_t given, int64_t* need, F call) {
  size_t bytes = size_t(given);
  int rc = call(ws, &bytes);
  if (rc == ZR_ERR_WORKSPACE && ws) {
    bytes = 0;
    if (call(nullptr, &bytes) == ZR_OK && bytes <= size_t(given)) return rc;  // misaligned
  }
  *need = int64_t(bytes);
  return rc;
}

}  // namespace

extern "C" {

int zr_packed_layer_norm_fwd(const int64_t* words) {
  if (!words) return ZR_ERR_NULL;
  Reader r{words};
  const double eps = r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  float* mean = r.ptr<float>();
  float* rstd = r.ptr<float>();
  const zr_tensor x = r.tensor(), gamma = r.tensor(), beta = r.tensor(), y = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  if (y.ndim != x.ndim) return ZR_ERR_SHAPE;
  return zr_layer_norm_fwd(dt, x, gamma, beta, float(eps), const_cast<void*>(y.data), y.strides, mean,
                           rstd, stream);
}

int zr_packed_layer_norm_bwd(const int64_t* words, int64_t* need) {
  if (!words || !need) return ZR_ERR_NULL;
  Reader r{words};
  r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  const float* mean = r.ptr<float>();
  const float* rstd = r.ptr<float>();
  void* gg = r.ptr<void>();
  void* gb = r.ptr<void>();
  void* ws = r.ptr<void>();
  const int64_t given = r.i64();
  const zr_tensor g = r.tensor(), x = r.tensor(), gamma = r.tensor(), gx = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  if (gx.data && gx.ndim != x.ndim) return ZR_ERR_SHAPE;
  return with_need(ws, given, need, [&](void* w, size_t* n) {
    return zr_layer_norm_bwd(dt, g, x, gamma, mean, rstd, const_cast<void*>(gx.data),
                             gx.data ? gx.strides : nullptr, gg, gb, w, n, stream);
  });
}

int zr_packed_dropout_fwd(const int64_t* words) {
  if (!words) return ZR_ERR_NULL;
  Reader r{words};
  const double p = r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  const uint64_t seed = uint64_t(r.i64()), offset = uint64_t(r.i64());
  const zr_rng rng{seed, offset, r.ptr<const uint64_t>()};
  const zr_tensor x = r.tensor(), residual = r.tensor(), out = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  if (out.ndim != x.ndim) return ZR_ERR_SHAPE;
  return zr_dropout_fwd(dt, x, residual, p, rng, const_cast<void*>(out.data), out.strides, stream);
}

int zr_packed_dropout_bwd(const int64_t* words) {
  if (!words) return ZR_ERR_NULL;
  Reader r{words};
  const double p = r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  const uint64_t seed = uint64_t(r.i64()), offset = uint64_t(r.i64());
  const zr_rng rng{seed, offset, r.ptr<const uint64_t>()};
  const zr_tensor g = r.tensor(), gx = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  if (gx.ndim != g.ndim) return ZR_ERR_SHAPE;
  return zr_dropout_bwd(dt, g, p, rng, const_cast<void*>(gx.data), gx.strides, stream);
}

int zr_packed_linear_xent_fwd(const int64_t* words, int64_t* need) {
  if (!words || !need) return ZR_ERR_NULL;
  Reader r{words};
  r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  const auto it = static_cast<zr_index>(r.i64());
  const int64_t ignore = r.i64();
  const auto red = static_cast<zr_reduction>(r.i64());
  float* loss = r.ptr<float>();
  float* lse = r.ptr<float>();
  void* ws = r.ptr<void>();
  const int64_t given = r.i64();
  const zr_tensor x = r.tensor(), w = r.tensor(), labels = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  return with_need(ws, given, need, [&](void* wp, size_t* n) {
    return zr_linear_xent_fwd(dt, x, w, it, labels, ignore, red, loss, lse, wp, n, stream);
  });
}

int zr_packed_linear_xent_bwd(const int64_t* words, int64_t* need) {
  if (!words || !need) return ZR_ERR_NULL;
  Reader r{words};
  r.real();
  const auto dt = static_cast<zr_dtype>(r.i64());
  const zr_stream_t stream = r.ptr<CUstream_st>();
  const auto it = static_cast<zr_index>(r.i64());
  const int64_t ignore = r.i64();
  const auto red = static_cast<zr_reduction>(r.i64());
  const float* grad_loss = r.ptr<float>();
  const float* lse = r.ptr<float>();
  void* gx = r.ptr<void>();
  void* gw = r.ptr<void>();
  void* ws = r.ptr<void>();
  const int64_t given = r.i64();
  const zr_tensor x = r.tensor(), w = r.tensor(), labels = r.tensor();
  if (!r.ok) return ZR_ERR_RANK;
  return with_need(ws, given, need, [&](void* wp, size_t* n) {
    return zr_linear_xent_bwd(dt, grad_loss, x, w, it, labels, ignore, red, lse, gx, gw, wp, n, stream);
  });
}

}  // extern "C"
