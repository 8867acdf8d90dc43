// zr_torch.cpp — CPython module that hands torch tensors to the training
// operators of include/zr.h: argument marshalling, output and workspace
// allocation, the current stream.  Their calls are short, so what the binding
// costs counts: built on the argument vector and the tensors' own size and
// stride arrays, a call does nothing per argument but read it (layer norm of
// one row on a Grace core: 41 us through ctypes structures, 6.6 here).
//
// Each function returns its tensors, or the zr_status of a failed call as an
// int (train.py raises it).  Wrong argument types raise here.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <memory>
#include <vector>

#include "../../include/zr.h"

namespace {

using at::Tensor;

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* fmt, const char* what) {
  PyErr_Format(type, fmt, what);
  throw Failed();
}

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

// An optional tensor argument.
const Tensor* maybe(PyObject* o, const char* what) {
  return o == Py_None ? nullptr : &tensor(o, what);
}

// The zr_dtype that every given tensor shares; all of them on a CUDA device.
zr_dtype dtype_of(std::initializer_list<const Tensor*> ts) {
  const auto dt = (*ts.begin())->scalar_type();
  if (dt != at::kFloat && dt != at::kBFloat16)
    fail(PyExc_TypeError, "zr operands must be float32 or bfloat16 (got %s)", c10::toString(dt));
  for (const Tensor* t : ts)
    if (t && t->scalar_type() != dt)
      fail(PyExc_TypeError, "operands mix element types (got %s)", c10::toString(t->scalar_type()));
  for (const Tensor* t : ts)
    if (t && !t->is_cuda()) fail(PyExc_ValueError, "zr operands must be CUDA tensors%s", "");
  return dt == at::kFloat ? ZR_F32 : ZR_BF16;
}

void same_shape(const Tensor& t, at::IntArrayRef shape, const char* what) {
  if (t.sizes() != shape) fail(PyExc_ValueError, "%s has the wrong shape", what);
}
void dense(const Tensor& t, at::IntArrayRef shape, const char* what) {
  same_shape(t, shape, what);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", what);
}
// A float32 CUDA tensor, dense over `shape`.
const float* stats(const Tensor& t, at::IntArrayRef shape, const char* what) {
  if (t.scalar_type() != at::kFloat) fail(PyExc_TypeError, "%s must be float32", what);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", what);
  dense(t, shape, what);
  return static_cast<const float*>(t.data_ptr());
}

const float* stats(PyObject* o, at::IntArrayRef shape, const char* what) {
  return stats(tensor(o, what), shape, what);
}

zr_tensor desc(const Tensor& t) {
  return {t.data_ptr(), int32_t(t.dim()), t.sizes().data(), t.strides().data()};
}
zr_tensor desc(const Tensor* t) { return t ? desc(*t) : zr_tensor{nullptr, 0, nullptr, nullptr}; }
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType dt) {
  return at::detail::empty_cuda(shape, dt, like.device(), c10::nullopt);
}
// The caller's output tensor, or a new contiguous one.
Tensor output(const Tensor* given, at::IntArrayRef shape, const Tensor& like, const char* what) {
  if (!given) return empty(shape, like, like.scalar_type());
  same_shape(*given, shape, what);
  return *given;
}

zr_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<zr_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... Ts>
PyObject* result(int rc, const Ts&... ts) {
  if (rc) return PyLong_FromLong(rc);
  if constexpr (sizeof...(Ts) == 1) return wrap(ts...);
  PyObject* tuple = PyTuple_New(sizeof...(Ts));
  if (!tuple) throw Failed();
  Py_ssize_t i = 0;
  ((PyTuple_SET_ITEM(tuple, i++, wrap(ts))), ...);
  return tuple;
}

// Runs call(workspace, &bytes) with the caller's workspace or, where that is
// missing or too small, with one of the size the call asks for.
template <typename F>
int with_workspace(const Tensor* given, const Tensor& like, F call) {
  size_t need = 0;
  int rc = call(nullptr, &need);
  if (rc) return rc;
  Tensor own;
  if (given && (given->scalar_type() != at::kByte || !given->is_cuda() || !given->is_contiguous()))
    fail(PyExc_TypeError, "%s must be a contiguous uint8 CUDA tensor", "workspace");
  if (need && (!given || size_t(given->numel()) < need)) {
    own = empty({int64_t(need > 16 ? need : 16)}, like, at::kByte);
    given = &own;
  }
  size_t bytes = given ? size_t(given->numel()) : 0;
  // Not NULL even where nothing is needed: that would ask for the size.
  void* ws = bytes ? given->data_ptr() : reinterpret_cast<void*>(uintptr_t(16));
  return call(ws, &bytes);
}

// The module's functions run with the GIL and turn C++ exceptions into Python
// ones.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    at::AutoDispatchBelowADInplaceOrView guard;
    return F(args, n);
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "wrong number of arguments%s", "");
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}
// Modulo 2^64.
uint64_t word(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Failed();
  const unsigned long long v = PyLong_AsUnsignedLongLongMask(i);
  Py_DECREF(i);
  if (v == ~0ull && PyErr_Occurred()) throw Failed();
  return v;
}

// x, gamma, beta, eps, out, keep_stats -> (y, mean, rstd)
PyObject* layer_norm_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  const Tensor& x = tensor(a[0], "x");
  const Tensor *gamma = maybe(a[1], "gamma"), *beta = maybe(a[2], "beta"), *out = maybe(a[4], "out");
  const double eps = real(a[3]);
  const zr_dtype dt = dtype_of({&x, gamma, beta, out});
  const Tensor y = output(out, x.sizes(), x, "out");
  Tensor mean, rstd;
  if (a[5] == Py_True) {
    const auto lead = x.dim() ? x.sizes().slice(0, x.dim() - 1) : x.sizes();
    mean = empty(lead, x, at::kFloat);
    rstd = empty(lead, x, at::kFloat);
  }
  const int rc = zr_layer_norm_fwd(dt, desc(x), desc(gamma), desc(beta), float(eps), y.data_ptr(),
                                   y.strides().data(), static_cast<float*>(ptr(mean)),
                                   static_cast<float*>(ptr(rstd)), stream_of(x));
  return result(rc, y, mean, rstd);
}

// grad_out, x, gamma, mean, rstd, want_x, want_gamma, want_beta, grad_x, grad_gamma, grad_beta,
// workspace -> (grad_x, grad_gamma, grad_beta)
PyObject* layer_norm_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 12);
  const Tensor &g = tensor(a[0], "grad_out"), &x = tensor(a[1], "x");
  const Tensor* gamma = maybe(a[2], "gamma");
  const Tensor *ox = maybe(a[8], "grad_x"), *og = maybe(a[9], "grad_gamma"), *ob = maybe(a[10], "grad_beta");
  const Tensor* ws = maybe(a[11], "workspace");
  const zr_dtype dt = dtype_of({&x, &g, gamma, ox, og, ob});
  const auto s = x.sizes();
  const auto lead = x.dim() ? s.slice(0, x.dim() - 1) : s;
  const auto width = x.dim() ? s.slice(x.dim() - 1, 1) : s;
  const float* mean = stats(a[3], lead, "mean");
  const float* rstd = stats(a[4], lead, "rstd");
  if (og) dense(*og, width, "grad_gamma");
  if (ob) dense(*ob, width, "grad_beta");
  Tensor gx, gg, gb;
  if (ox || a[5] == Py_True) gx = output(ox, s, x, "grad_x");
  if (og || a[6] == Py_True) gg = output(og, width, x, "grad_gamma");
  if (ob || a[7] == Py_True) gb = output(ob, width, x, "grad_beta");
  const zr_stream_t st = stream_of(x);
  const int rc = with_workspace(ws, x, [&](void* w, size_t* bytes) {
    return zr_layer_norm_bwd(dt, desc(g), desc(x), desc(gamma), mean, rstd, ptr(gx),
                             gx.defined() ? gx.strides().data() : nullptr, ptr(gg), ptr(gb), w, bytes, st);
  });
  return result(rc, gx, gg, gb);
}

zr_rng rng_of(PyObject* seed, PyObject* offset, PyObject* device_offset) {
  zr_rng r{word(seed), word(offset), nullptr};
  if (device_offset != Py_None) {
    const Tensor& t = tensor(device_offset, "device_offset");
    if (t.scalar_type() != at::kLong || t.numel() != 1)
      fail(PyExc_TypeError, "%s must be one int64 element", "device_offset");
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", "device_offset");
    r.device_offset = static_cast<const uint64_t*>(t.data_ptr());
  }
  return r;
}

// x, p, seed, offset, residual, out, device_offset -> out
PyObject* dropout_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 7);
  const Tensor& x = tensor(a[0], "x");
  const double p = real(a[1]);
  const zr_rng rng = rng_of(a[2], a[3], a[6]);
  const Tensor *residual = maybe(a[4], "residual"), *out = maybe(a[5], "out");
  if (residual) same_shape(*residual, x.sizes(), "residual");
  const zr_dtype dt = dtype_of({&x, residual, out});
  const Tensor y = output(out, x.sizes(), x, "out");
  const int rc = zr_dropout_fwd(dt, desc(x), desc(residual), p, rng, y.data_ptr(), y.strides().data(),
                                stream_of(x));
  return result(rc, y);
}

// grad_out, p, seed, offset, grad_x, device_offset -> grad_x
PyObject* dropout_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  const Tensor& g = tensor(a[0], "grad_out");
  const double p = real(a[1]);
  const zr_rng rng = rng_of(a[2], a[3], a[5]);
  const Tensor* out = maybe(a[4], "grad_x");
  const zr_dtype dt = dtype_of({&g, out});
  const Tensor gx = output(out, g.sizes(), g, "grad_x");
  const int rc = zr_dropout_bwd(dt, desc(g), p, rng, gx.data_ptr(), gx.strides().data(), stream_of(g));
  return result(rc, gx);
}

zr_index label_type(const Tensor& labels, at::IntArrayRef lead) {
  const auto dt = labels.scalar_type();
  if (dt != at::kLong && dt != at::kInt) fail(PyExc_TypeError, "%s must be int32 or int64", "labels");
  if (!labels.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", "labels");
  same_shape(labels, lead, "labels");
  return dt == at::kLong ? ZR_I64 : ZR_I32;
}

// x, w, labels, reduction code, ignore_index, workspace -> (loss, lse)
PyObject* linear_xent_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &labels = tensor(a[2], "labels");
  const auto red = static_cast<zr_reduction>(integer(a[3]));
  const int64_t ignore = integer(a[4]);
  const Tensor* ws = maybe(a[5], "workspace");
  const zr_dtype dt = dtype_of({&x, &w});
  const auto lead = x.dim() ? x.sizes().slice(0, x.dim() - 1) : x.sizes();
  const zr_index it = label_type(labels, lead);
  const Tensor loss = empty(red == ZR_NONE ? lead : at::IntArrayRef(), x, at::kFloat);
  const Tensor lse = empty(lead, x, at::kFloat);
  const zr_stream_t st = stream_of(x);
  const int rc = with_workspace(ws, x, [&](void* wp, size_t* bytes) {
    return zr_linear_xent_fwd(dt, desc(x), desc(w), it, desc(labels), ignore, red,
                              static_cast<float*>(ptr(loss)), static_cast<float*>(ptr(lse)), wp, bytes, st);
  });
  return result(rc, loss, lse);
}

// grad_loss, x, w, labels, lse, reduction code, ignore_index, want_x, want_w, grad_x, grad_w,
// workspace -> (grad_x, grad_w)
PyObject* linear_xent_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 12);
  const Tensor &given = tensor(a[0], "grad_loss"), &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
  const Tensor& labels = tensor(a[3], "labels");
  const auto red = static_cast<zr_reduction>(integer(a[5]));
  const int64_t ignore = integer(a[6]);
  const Tensor *ox = maybe(a[9], "grad_x"), *ow = maybe(a[10], "grad_w"), *ws = maybe(a[11], "workspace");
  const zr_dtype dt = dtype_of({&x, &w, ox, ow});
  const auto lead = x.dim() ? x.sizes().slice(0, x.dim() - 1) : x.sizes();
  const zr_index it = label_type(labels, lead);
  const float* lse = stats(a[4], lead, "lse");
  // A view, as loss.sum() hands down an expanded one, is copied: one float per row.
  const Tensor gl = given.contiguous();
  const float* grad_loss = stats(gl, gl.sizes(), "grad_loss");
  if (gl.numel() != (red == ZR_NONE ? labels.numel() : 1))
    fail(PyExc_ValueError, "%s has the wrong number of elements", "grad_loss");
  if (ox) dense(*ox, x.sizes(), "grad_x");
  if (ow) dense(*ow, w.sizes(), "grad_w");
  Tensor gx, gw;
  if (ox || a[7] == Py_True) gx = output(ox, x.sizes(), x, "grad_x");
  if (ow || a[8] == Py_True) gw = output(ow, w.sizes(), w, "grad_w");
  const zr_stream_t st = stream_of(x);
  const int rc = with_workspace(ws, x, [&](void* wp, size_t* bytes) {
    return zr_linear_xent_bwd(dt, grad_loss, desc(x), desc(w), it, desc(labels), ignore, red, lse,
                              ptr(gx), ptr(gw), wp, bytes, st);
  });
  return result(rc, gx, gw);
}

// The scale argument, D^-1/2 where it is None.
float scale_of(PyObject* o, const Tensor& q) {
  if (o != Py_None) return float(real(o));
  return q.dim() && q.size(-1) > 0 ? float(1.0 / std::sqrt(double(q.size(-1)))) : 1.f;
}
struct Offsets {
  const int32_t* p = nullptr;
  int32_t sequences = 0;
};
Offsets offsets_of(PyObject* o, const Tensor& q) {
  if (o == Py_None) return {};
  const Tensor& t = tensor(o, "offsets");
  if (t.scalar_type() != at::kInt) fail(PyExc_TypeError, "%s must be int32", "offsets");
  if (!t.is_cuda() || t.device() != q.device()) fail(PyExc_ValueError, "%s must be on the operands' device", "offsets");
  if (t.dim() != 1 || t.numel() < 1 || t.numel() > (int64_t(1) << 30) || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be a contiguous vector of at least one border", "offsets");
  return {static_cast<const int32_t*>(t.data_ptr()), int32_t(t.numel() - 1)};
}

// q, k, v, scale, offsets, out, keep_lse, keep_low, workspace -> (out, lse, low)
PyObject* attention_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 9);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const Tensor *out = maybe(a[5], "out"), *ws = maybe(a[8], "workspace");
  const zr_dtype dt = dtype_of({&q, &k, &v, out});
  const float scale = scale_of(a[3], q);
  const Offsets off = offsets_of(a[4], q);
  const Tensor y = output(out, q.sizes(), q, "out");
  Tensor lse, low;
  if (PyObject_IsTrue(a[6]) == 1) lse = empty(q.dim() ? q.sizes().slice(0, q.dim() - 1) : q.sizes(), q, at::kFloat);
  if (PyObject_IsTrue(a[7]) == 1 && dt == ZR_BF16) low = empty(q.sizes(), q, at::kBFloat16);
  const zr_stream_t st = stream_of(q);
  const int rc = with_workspace(ws, q, [&](void* w, size_t* bytes) {
    return zr_attention_fwd(dt, desc(q), desc(k), desc(v), scale, off.p, off.sequences, y.data_ptr(), y.strides().data(),
                            ptr(low), static_cast<float*>(ptr(lse)), w, bytes, st);
  });
  return result(rc, y, lse, low);
}

// grad_out, q, k, v, out, lse, low, scale, offsets, want_q, want_k, want_v, grad_q, grad_k, grad_v,
// workspace -> (grad_q, grad_k, grad_v)
PyObject* attention_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 16);
  const Tensor &g = tensor(a[0], "grad_out"), &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const Tensor& o = tensor(a[4], "out");
  const Tensor *low = maybe(a[6], "low"), *oq = maybe(a[12], "grad_q"), *ok = maybe(a[13], "grad_k"), *ov = maybe(a[14], "grad_v");
  const Tensor* ws = maybe(a[15], "workspace");
  const zr_dtype dt = dtype_of({&q, &k, &v, &g, &o, low, oq, ok, ov});
  const float* lse = stats(a[5], q.dim() ? q.sizes().slice(0, q.dim() - 1) : q.sizes(), "lse");
  if (low) dense(*low, q.sizes(), "low");
  const float scale = scale_of(a[7], q);
  const Offsets off = offsets_of(a[8], q);
  Tensor gq, gk, gv;
  if (oq || a[9] == Py_True) gq = output(oq, q.sizes(), q, "grad_q");
  if (ok || a[10] == Py_True) gk = output(ok, k.sizes(), q, "grad_k");
  if (ov || a[11] == Py_True) gv = output(ov, v.sizes(), q, "grad_v");
  const auto strides = [](const Tensor& t) { return t.defined() ? t.strides().data() : nullptr; };
  const zr_stream_t st = stream_of(q);
  const int rc = with_workspace(ws, q, [&](void* w, size_t* bytes) {
    return zr_attention_bwd(dt, desc(g), desc(q), desc(k), desc(v), desc(o), low ? low->data_ptr() : nullptr, lse,
                            scale, off.p, off.sequences, ptr(gq), strides(gq), ptr(gk), strides(gk), ptr(gv),
                            strides(gv), w, bytes, st);
  });
  return result(rc, gq, gk, gv);
}

// part, interleaved, base, factor, original, low, high, magnitude -> the plan's bytes
PyObject* rotary_plan(PyObject* const* a, Py_ssize_t n) {
  count(n, 8);
  zr_rotary plan;
  const int64_t part = integer(a[0]);
  const int rc = zr_rotary_plan(part < 0 || part > (1 << 30) ? -1 : int32_t(part), PyObject_IsTrue(a[1]) == 1, real(a[2]),
                                real(a[3]), real(a[4]), real(a[5]), real(a[6]), real(a[7]), &plan);
  if (rc) return PyLong_FromLong(rc);
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&plan), sizeof plan);
}

// x, plan, positions, start, out, backward -> out
PyObject* rotary(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  const Tensor& x = tensor(a[0], "x");
  if (!PyBytes_Check(a[1]) || PyBytes_GET_SIZE(a[1]) != Py_ssize_t(sizeof(zr_rotary)))
    fail(PyExc_TypeError, "%s must come from zr_rotary_plan", "plan");
  zr_rotary plan;
  std::memcpy(&plan, PyBytes_AS_STRING(a[1]), sizeof plan);
  const Tensor *positions = maybe(a[2], "positions"), *out = maybe(a[4], "out");
  const int64_t start = integer(a[3]);
  const zr_dtype dt = dtype_of({&x, out});
  zr_index type = ZR_I64;
  if (positions) {
    const auto pt = positions->scalar_type();
    if (pt != at::kLong && pt != at::kInt) fail(PyExc_TypeError, "%s must be int32 or int64", "positions");
    if (!positions->is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", "positions");
    if (x.dim() >= 2) same_shape(*positions, x.sizes().slice(0, x.dim() - 2), "positions");
    type = pt == at::kLong ? ZR_I64 : ZR_I32;
  }
  const Tensor y = output(out, x.sizes(), x, "out");
  const int rc = (a[5] == Py_True ? zr_rotary_bwd : zr_rotary_fwd)(dt, desc(x), &plan, type, desc(positions), start,
                                                                   y.data_ptr(), y.strides().data(), stream_of(x));
  return result(rc, y);
}

// The items of a list or tuple.
struct Items {
  PyObject* fast;
  Items(PyObject* o, const char* what) : fast(PySequence_Fast(o, what)) {
    if (!fast) throw Failed();
  }
  Items(const Items&) = delete;
  ~Items() { Py_DECREF(fast); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// The data of a contiguous CUDA tensor of `numel` elements on `like`'s device.
void* flat(const Tensor& t, at::ScalarType dt, int64_t numel, const Tensor& like, const char* what) {
  if (t.scalar_type() != dt) {
    PyErr_Format(PyExc_TypeError, "%s must be %s", what, c10::toString(dt));
    throw Failed();
  }
  if (!t.is_cuda() || t.device() != like.device()) fail(PyExc_ValueError, "%s must be CUDA tensors of one device", what);
  if (t.numel() != numel) fail(PyExc_ValueError, "%s has the wrong number of elements", what);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", what);
  return t.data_ptr();
}
void* flat(PyObject* o, at::ScalarType dt, int64_t numel, const Tensor& like, const char* what) {
  return flat(tensor(o, what), dt, numel, like, what);
}
int64_t blocks_of(int64_t n) { return (n + ZR_ADAMW_BLOCK - 1) / ZR_ADAMW_BLOCK; }
const void* one(PyObject* o, at::ScalarType dt, const Tensor& like, const char* what) {
  return o == Py_None ? nullptr : flat(o, dt, 1, like, what);
}

// params, grads, ms, vs, step, lr, beta1, beta2, eps, weight_decay, copies, m_scales, v_scales, seed,
// device_step, device_lr, grad_scale -> the status
PyObject* adamw_step(PyObject* const* a, Py_ssize_t n) {
  count(n, 17);
  const Items params(a[0], "params must be a sequence"), grads(a[1], "grads must be a sequence"),
      ms(a[2], "ms must be a sequence"), vs(a[3], "vs must be a sequence");
  const Py_ssize_t k = params.size();
  const auto same = [&](const Items& x, const char* what) {
    if (x.size() != k) fail(PyExc_ValueError, "%s must have one entry per parameter", what);
  };
  const auto optional = [&](PyObject* o, const char* what) {
    std::unique_ptr<Items> x;
    if (o != Py_None) {
      x = std::make_unique<Items>(o, what);
      same(*x, what);
    }
    return x;
  };
  same(grads, "grads");
  same(ms, "ms");
  same(vs, "vs");
  const bool decays = !PyNumber_Check(a[9]);
  const auto wd = decays ? optional(a[9], "weight_decay") : nullptr;
  const double decay = decays ? 0 : real(a[9]);
  const auto copies = optional(a[10], "copies"), msc = optional(a[11], "m_scales"), vsc = optional(a[12], "v_scales");
  if (!msc != !vsc) fail(PyExc_ValueError, "%s come together", "m_scales and v_scales");
  if (k > 0x7FFFFFFF) fail(PyExc_ValueError, "too many tensors%s", "");
  zr_adamw how{};
  how.step = integer(a[4]);
  how.lr = real(a[5]);
  how.beta1 = real(a[6]);
  how.beta2 = real(a[7]);
  how.eps = real(a[8]);
  how.seed = word(a[13]);
  std::vector<zr_adamw_tensor> list(size_t(k), zr_adamw_tensor{});
  auto gt = at::kFloat;
  const auto st = msc ? at::kByte : at::kFloat;
  zr_stream_t stream = nullptr;
  for (Py_ssize_t i = 0; i < k; ++i) {
    const Tensor& p = tensor(params[i], "params");
    const Tensor& g = tensor(grads[i], "grads");
    if (i == 0) {
      gt = g.scalar_type();
      if (gt != at::kFloat && gt != at::kBFloat16) fail(PyExc_TypeError, "%s must be float32 or bfloat16", "grads");
      if (!p.is_cuda()) fail(PyExc_ValueError, "%s must be CUDA tensors", "params");
      stream = stream_of(p);
      how.device_step = static_cast<const int64_t*>(one(a[14], at::kLong, p, "device_step"));
      how.device_lr = static_cast<const float*>(one(a[15], at::kFloat, p, "device_lr"));
      how.device_grad_scale = static_cast<const float*>(one(a[16], at::kFloat, p, "grad_scale"));
    }
    const Tensor& first = tensor(params[0], "params");
    const int64_t m = p.numel();
    zr_adamw_tensor& t = list[size_t(i)];
    t.n = m;
    t.param = static_cast<float*>(flat(p, at::kFloat, m, first, "params"));
    t.grad = flat(g, gt, m, first, "grads");
    t.m = flat(ms[i], st, m, first, "ms");
    t.v = flat(vs[i], st, m, first, "vs");
    if (copies && (*copies)[i] != Py_None) t.copy = flat((*copies)[i], at::kBFloat16, m, first, "copies");
    if (msc) {
      t.m_scale = static_cast<float*>(flat((*msc)[i], at::kFloat, blocks_of(m), first, "m_scales"));
      t.v_scale = static_cast<float*>(flat((*vsc)[i], at::kFloat, blocks_of(m), first, "v_scales"));
    }
    t.weight_decay = float(wd ? real((*wd)[i]) : decay);
  }
  return PyLong_FromLong(zr_adamw_step(gt == at::kBFloat16 ? ZR_BF16 : ZR_F32, msc ? 8 : 32, int32_t(k), list.data(), &how, stream));
}

// ms, vs, m_scales, v_scales, out (None, or two sequences) -> (m values, v values), or out
PyObject* adamw_state(PyObject* const* a, Py_ssize_t n) {
  count(n, 5);
  const Items ms(a[0], "ms must be a sequence"), vs(a[1], "vs must be a sequence"),
      msc(a[2], "m_scales must be a sequence"), vsc(a[3], "v_scales must be a sequence");
  const Py_ssize_t k = ms.size();
  if (vs.size() != k || msc.size() != k || vsc.size() != k)
    fail(PyExc_ValueError, "%s must have as many entries", "vs, m_scales and v_scales");
  std::unique_ptr<Items> out[2];
  if (a[4] != Py_None) {
    const Items both(a[4], "out must hold two sequences");
    if (both.size() != 2) fail(PyExc_ValueError, "%s must hold two sequences", "out");
    for (int i = 0; i < 2; ++i) {
      out[i] = std::make_unique<Items>(both[i], "out must hold two sequences");
      if (out[i]->size() != k) fail(PyExc_ValueError, "%s must have as many entries", "out");
    }
  }
  std::vector<zr_adamw_tensor> list(size_t(k), zr_adamw_tensor{});
  std::vector<void*> to[2];
  std::vector<Tensor> made[2];  // where no out is given
  zr_stream_t stream = nullptr;
  for (Py_ssize_t i = 0; i < k; ++i) {
    const Tensor &m = tensor(ms[i], "ms"), &first = tensor(ms[0], "ms");
    if (i == 0) {
      if (!m.is_cuda()) fail(PyExc_ValueError, "%s must be CUDA tensors", "ms");
      stream = stream_of(m);
    }
    zr_adamw_tensor& t = list[size_t(i)];
    t.n = m.numel();
    t.m = flat(m, at::kByte, t.n, first, "ms");
    t.v = flat(vs[i], at::kByte, t.n, first, "vs");
    t.m_scale = static_cast<float*>(flat(msc[i], at::kFloat, blocks_of(t.n), first, "m_scales"));
    t.v_scale = static_cast<float*>(flat(vsc[i], at::kFloat, blocks_of(t.n), first, "v_scales"));
    for (int j = 0; j < 2; ++j) {
      if (!out[j]) made[j].push_back(empty(m.sizes(), m, at::kBFloat16));
      to[j].push_back(flat(out[j] ? tensor((*out[j])[i], "out") : made[j].back(), at::kBFloat16, t.n, first, "out"));
    }
  }
  const int rc = zr_adamw_state(int32_t(k), list.data(), to[0].data(), to[1].data(), stream);
  if (rc) return PyLong_FromLong(rc);
  if (a[4] != Py_None) {
    Py_INCREF(a[4]);
    return a[4];
  }
  PyObject* both = PyTuple_New(2);
  if (!both) throw Failed();
  for (int j = 0; j < 2; ++j) {
    PyObject* l = PyList_New(k);
    if (!l) {
      Py_DECREF(both);
      throw Failed();
    }
    for (Py_ssize_t i = 0; i < k; ++i) PyList_SET_ITEM(l, i, wrap(made[j][size_t(i)]));
    PyTuple_SET_ITEM(both, j, l);
  }
  return both;
}

#define ZR_METHOD(F) {#F, reinterpret_cast<PyCFunction>(entry<F>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ZR_METHOD(layer_norm_fwd),  ZR_METHOD(layer_norm_bwd),
                         ZR_METHOD(dropout_fwd),     ZR_METHOD(dropout_bwd),
                         ZR_METHOD(linear_xent_fwd), ZR_METHOD(linear_xent_bwd),
                         ZR_METHOD(attention_fwd),   ZR_METHOD(attention_bwd),
                         ZR_METHOD(rotary_plan),     ZR_METHOD(rotary),
                         ZR_METHOD(adamw_step),      ZR_METHOD(adamw_state),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "zr_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_zr_torch(void) { return PyModule_Create(&module); }
