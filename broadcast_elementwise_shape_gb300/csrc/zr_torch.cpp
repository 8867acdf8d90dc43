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
  if (!given || size_t(given->numel()) < need) {
    own = empty({int64_t(need > 16 ? need : 16)}, like, at::kByte);
    given = &own;
  }
  size_t bytes = size_t(given->numel());
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

#define ZR_METHOD(F) {#F, reinterpret_cast<PyCFunction>(entry<F>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ZR_METHOD(layer_norm_fwd),  ZR_METHOD(layer_norm_bwd),
                         ZR_METHOD(dropout_fwd),     ZR_METHOD(dropout_bwd),
                         ZR_METHOD(linear_xent_fwd), ZR_METHOD(linear_xent_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "zr_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_zr_torch(void) { return PyModule_Create(&module); }
