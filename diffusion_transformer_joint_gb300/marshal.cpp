// The argument marshalling of binding.py for its 8-bit products and its
// cross-attention, compiled: the same calls into libflux_attn.so with the same
// checks of types, shapes, devices and strides. A call that passes them is made
// here (some 1 us beside the launch; in Python they take 5 to 9); any other one
// returns None, and binding.py, which goes through the checks again, says what is
// wrong with it. Nothing is kept from one call for another but the addresses of the
// library's functions and status words.
//
// C++ exceptions end here (also as None): a tensor without memory or strides, say.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>

#include <cstdint>

#include "flux_attn.h"

namespace {

decltype(&flux_quantize_fp8) quantize_fn;
decltype(&flux_linear_fp8) linear_fn;
decltype(&flux_cross_attention) cross_fn;
constexpr int kMaxDevices = 64;
int32_t *own_words[kMaxDevices];  // the library's status words

using at::Tensor;

const Tensor *tensor(PyObject *o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}
bool absent(PyObject *o) { return o == Py_None; }
bool on(const Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// [B, S, width] or [S, width] with contiguous channels.
struct Rows {
  void *p = nullptr;
  int64_t bs = 0, rs = 0;
};
bool take_rows(const Tensor *t, bool batched, int64_t B, int64_t S, int64_t width,
               at::ScalarType type, int dev, Rows &r) {
  const int64_t n = batched ? 3 : 2;
  if (t == nullptr || t->scalar_type() != type || t->dim() != n || !on(*t, dev)) return false;
  const auto sizes = t->sizes(), strides = t->strides();
  if ((batched && sizes[0] != B) || sizes[n - 2] != S || sizes[n - 1] != width) return false;
  if (strides[n - 1] != 1) return false;
  r.p = const_cast<void *>(t->const_data_ptr());
  r.bs = batched ? strides[0] : 0;
  r.rs = strides[n - 2];
  return true;
}

// [width], or [1, width] or [B, width]: one vector, or one per batch element.
bool take_vector(const Tensor *t, int64_t B, int64_t width, at::ScalarType type, int dev,
                 const void *&p, int64_t &bs) {
  if (t == nullptr || t->scalar_type() != type || !on(*t, dev)) return false;
  const int64_t n = t->dim();
  if (n < 1 || n > 2 || t->size(n - 1) != width || (width > 1 && t->stride(n - 1) != 1)) return false;
  if (n == 2 && t->size(0) != 1 && t->size(0) != B) return false;
  p = t->const_data_ptr();
  bs = n == 2 && t->size(0) == B && B > 1 ? t->stride(0) : 0;
  return true;
}

// fp32 [B, R, G] ([R, G]) of any strides.
struct Scales {
  float *p = nullptr;
  int64_t bs = 0, rs = 0, ks = 0;
};
bool take_scales(const Tensor *t, bool batched, int64_t B, int64_t R, int64_t G, int dev, Scales &s) {
  const int64_t n = batched ? 3 : 2;
  if (t == nullptr || t->scalar_type() != at::kFloat || t->dim() != n || !on(*t, dev)) return false;
  if ((batched && t->size(0) != B) || t->size(n - 2) != R || t->size(n - 1) != G) return false;
  s.p = static_cast<float *>(const_cast<void *>(t->const_data_ptr()));
  s.bs = batched ? t->stride(0) : 0;
  s.rs = t->stride(n - 2);
  s.ks = t->stride(n - 1);
  return true;
}

bool take_status(PyObject *o, int dev, int32_t *&p) {
  if (absent(o)) {
    p = own_words[dev];
    return p != nullptr;
  }
  const Tensor *t = tensor(o);
  if (t == nullptr || t->scalar_type() != at::kInt || t->numel() < 1 || !on(*t, dev)) return false;
  p = static_cast<int32_t *>(const_cast<void *>(t->const_data_ptr()));
  return true;
}

bool current(const Tensor *t, int &dev, void *&stream) {
  if (t == nullptr || !t->is_cuda()) return false;
  dev = t->get_device();
  if (dev < 0 || dev >= kMaxDevices || dev != c10::cuda::current_device()) return false;
  stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  return true;
}

int activation(PyObject *o) {
  if (absent(o)) return FLUX_ACT_NONE;
  if (!PyUnicode_Check(o)) return -1;
  if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return FLUX_ACT_SILU;
  if (PyUnicode_CompareWithASCIIString(o, "gelu_tanh") == 0) return FLUX_ACT_GELU_TANH;
  if (PyUnicode_CompareWithASCIIString(o, "swiglu") == 0) return FLUX_ACT_SWIGLU;
  return -1;
}

bool fits_int(int64_t v) { return v <= 0x7FFFFFFF; }

// The given output, or a new one: a reference of the caller's.
PyObject *given_or(PyObject *o, const Tensor &made) {
  if (absent(o)) return THPVariable_Wrap(made);
  Py_INCREF(o);
  return o;
}

// quantize_fp8(x, rows, out, scale) -> (out, scale), a status, or None
PyObject *quantize(PyObject *const *a) {
  const Tensor *x = tensor(a[0]);
  int dev;
  void *stream;
  if (!current(x, dev, stream) || !PyLong_Check(a[1])) return nullptr;
  const long rows = PyLong_AsLong(a[1]);
  const int64_t n = x->dim();
  if ((n != 2 && n != 3) || (rows != 1 && rows != 128) || (rows == 128 && n != 2)) return nullptr;
  const bool batched = n == 3, f32 = x->scalar_type() == at::kFloat;
  const int64_t B = batched ? x->size(0) : 1, S = x->size(n - 2), K = x->size(n - 1);
  if (!fits_int(B) || !fits_int(K) || B < 1 || S < 1 || K < 1) return nullptr;
  const int64_t G = (K + 127) / 128, R = rows == 1 ? S : (S + 127) / 128;
  Rows rx, rq;
  Scales sc;
  if (!take_rows(x, batched, B, S, K, f32 ? at::kFloat : at::kBFloat16, dev, rx)) return nullptr;
  Tensor out, scale;
  if (absent(a[2])) out = at::empty(x->sizes(), x->options().dtype(at::kFloat8_e4m3fn));
  if (absent(a[3])) {
    const auto opt = x->options().dtype(at::kFloat);
    if (rows == 128)
      scale = at::empty({R, G}, opt);
    else if (batched)
      scale = at::empty_strided({B, S, G}, {S, 1, B * S}, opt);
    else
      scale = at::empty_strided({S, G}, {1, S}, opt);
  }
  const Tensor *q = absent(a[2]) ? &out : tensor(a[2]);
  const Tensor *s = absent(a[3]) ? &scale : tensor(a[3]);
  if (!take_rows(q, batched, B, S, K, at::kFloat8_e4m3fn, dev, rq) ||
      !take_scales(s, batched, B, R, G, dev, sc))
    return nullptr;
  const int rc = quantize_fn(rx.p, rx.bs, rx.rs, f32 ? 1 : 0, static_cast<int>(B), S,
                             static_cast<int>(K), static_cast<int>(rows), rq.p, rq.bs, rq.rs, sc.p,
                             sc.bs, sc.rs, sc.ks, stream);
  if (rc != FLUX_OK) return PyLong_FromLong(rc);
  PyObject *o = given_or(a[2], out), *p = given_or(a[3], scale);
  PyObject *both = o != nullptr && p != nullptr ? PyTuple_Pack(2, o, p) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(p);
  return both;
}

// linear_fp8(x, x_scale, w, w_scale, bias, act, gate, residual, out, status)
PyObject *linear(PyObject *const *a) {
  const Tensor *x = tensor(a[0]), *w = tensor(a[2]);
  int dev;
  void *stream;
  const int act = activation(a[5]);
  if (act < 0 || w == nullptr || !current(x, dev, stream)) return nullptr;
  const int64_t n = x->dim();
  if ((n != 2 && n != 3) || w->dim() != 2) return nullptr;
  const bool batched = n == 3;
  const int64_t B = batched ? x->size(0) : 1, S = x->size(n - 2), K = x->size(n - 1);
  const int64_t rows = w->size(0), N = act == FLUX_ACT_SWIGLU ? rows / 2 : rows;
  if (!fits_int(B) || !fits_int(K) || B < 1 || S < 1 || K < 1 || N < 1) return nullptr;
  if (act == FLUX_ACT_SWIGLU && rows % 2 != 0) return nullptr;
  const int64_t G = (K + 127) / 128;
  Rows rx, rw, rr, ro;
  Scales sx, sw;
  if (!take_rows(x, batched, B, S, K, at::kFloat8_e4m3fn, dev, rx) ||
      !take_scales(tensor(a[1]), batched, B, S, G, dev, sx) ||
      !take_rows(w, false, 1, rows, K, at::kFloat8_e4m3fn, dev, rw) ||
      !take_scales(tensor(a[3]), false, 1, (rows + 127) / 128, G, dev, sw))
    return nullptr;
  if (!absent(a[7]) && !take_rows(tensor(a[7]), batched, B, S, N, at::kBFloat16, dev, rr))
    return nullptr;
  const void *bias = nullptr, *gate = nullptr;
  int64_t bias_bs = 0, gate_bs = 0;
  int vec_f32 = 0;
  if (!absent(a[4]) || !absent(a[6])) {
    const Tensor *one = tensor(absent(a[4]) ? a[6] : a[4]);
    if (one == nullptr) return nullptr;
    const auto type = one->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) return nullptr;
    vec_f32 = type == at::kFloat ? 1 : 0;
    if (!absent(a[4]) && !take_vector(tensor(a[4]), 1, rows, type, dev, bias, bias_bs)) return nullptr;
    if (!absent(a[6]) && !take_vector(tensor(a[6]), B, N, type, dev, gate, gate_bs)) return nullptr;
  }
  int32_t *status;
  if (!take_status(a[9], dev, status)) return nullptr;
  Tensor out;
  if (absent(a[8])) {
    const auto opt = x->options().dtype(at::kBFloat16);
    out = batched ? at::empty({B, S, N}, opt) : at::empty({S, N}, opt);
  }
  if (!take_rows(absent(a[8]) ? &out : tensor(a[8]), batched, B, S, N, at::kBFloat16, dev, ro))
    return nullptr;
  const int rc = linear_fn(rx.p, rx.bs, rx.rs, sx.p, sx.bs, sx.rs, sx.ks, rw.p, rw.rs, sw.p, sw.rs,
                           sw.ks, static_cast<int>(B), S, static_cast<int>(K), N, act, bias, gate,
                           gate_bs, vec_f32, rr.p, rr.bs, rr.rs, ro.p, ro.bs, ro.rs, status, stream);
  return rc != FLUX_OK ? PyLong_FromLong(rc) : given_or(a[8], out);
}

// Heads [B, S, H, D], a token's heads adjacent.
bool take_heads(const Tensor *t, int64_t B, int64_t S, int64_t H, int64_t D, int dev, Rows &r) {
  if (t == nullptr || t->scalar_type() != at::kBFloat16 || t->dim() != 4 || !on(*t, dev)) return false;
  const auto sizes = t->sizes(), strides = t->strides();
  if (sizes[0] != B || sizes[1] != S || sizes[2] != H || sizes[3] != D) return false;
  if (strides[3] != 1 || (H > 1 && strides[2] != D)) return false;
  r.p = const_cast<void *>(t->const_data_ptr());
  r.bs = strides[0];
  r.rs = strides[1];
  return true;
}

// cross_attention(q, k, v, lengths, mask, scale, out, status)
PyObject *cross(PyObject *const *a) {
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]);
  int dev;
  void *stream;
  if (!current(q, dev, stream) || k == nullptr || q->dim() != 4 || k->dim() != 4) return nullptr;
  const int64_t B = q->size(0), Sq = q->size(1), H = q->size(2), D = q->size(3);
  const int64_t Sk = k->size(1), Hk = k->size(2);
  if (!fits_int(B) || !fits_int(H) || !fits_int(Hk) || !fits_int(D)) return nullptr;
  Rows rq, rk, rv, ro;
  if (!take_heads(q, B, Sq, H, D, dev, rq) || !take_heads(k, B, Sk, Hk, D, dev, rk) ||
      !take_heads(tensor(a[2]), B, Sk, Hk, D, dev, rv))
    return nullptr;
  const int32_t *lengths = nullptr;
  const uint8_t *mask = nullptr;
  int64_t mask_bs = 0;
  if (!absent(a[3])) {
    const Tensor *t = tensor(a[3]);
    if (t == nullptr || t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != B ||
        !on(*t, dev) || !t->is_contiguous())
      return nullptr;
    lengths = static_cast<const int32_t *>(t->const_data_ptr());
  }
  if (!absent(a[4])) {
    const Tensor *t = tensor(a[4]);
    if (t == nullptr || (t->scalar_type() != at::kBool && t->scalar_type() != at::kByte) ||
        t->dim() != 2 || t->size(0) != B || t->size(1) != Sk || !on(*t, dev) ||
        (Sk > 1 && t->stride(1) != 1))
      return nullptr;
    mask = static_cast<const uint8_t *>(t->const_data_ptr());
    mask_bs = B > 1 ? t->stride(0) : 0;
  }
  float scale = 0.f;  // (the library's default)
  if (!absent(a[5])) {
    if (!PyFloat_Check(a[5])) return nullptr;
    const double given = PyFloat_AS_DOUBLE(a[5]);
    if (!(given <= 0x1p127)) return nullptr;
    scale = static_cast<float>(given);
    if (!(scale > 0.f)) return nullptr;
  }
  int32_t *status;
  if (!take_status(a[7], dev, status)) return nullptr;
  Tensor out;
  if (absent(a[6])) out = at::empty({B, Sq, H, D}, q->options());
  if (!take_heads(absent(a[6]) ? &out : tensor(a[6]), B, Sq, H, D, dev, ro)) return nullptr;
  const int rc = cross_fn(rq.p, rq.bs, rq.rs, rk.p, rk.bs, rk.rs, rv.p, rv.bs, rv.rs, lengths, mask,
                          mask_bs, static_cast<int>(B), Sq, Sk, static_cast<int>(H),
                          static_cast<int>(Hk), static_cast<int>(D), scale, ro.p, ro.bs,
                          ro.rs, status, stream);
  return rc != FLUX_OK ? PyLong_FromLong(rc) : given_or(a[6], out);
}

// fn's answer; None where a check failed or C++ threw.
template <PyObject *(*fn)(PyObject *const *), int kArgs>
PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n) {
  PyObject *r = nullptr;
  try {
    if (n == kArgs) r = fn(a);
  } catch (...) {
    r = nullptr;
  }
  if (r != nullptr) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// bind(quantize, linear, cross): addresses of the library's functions
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long q, l, c;
  if (!PyArg_ParseTuple(args, "KKK", &q, &l, &c)) return nullptr;
  quantize_fn = reinterpret_cast<decltype(quantize_fn)>(q);
  linear_fn = reinterpret_cast<decltype(linear_fn)>(l);
  cross_fn = reinterpret_cast<decltype(cross_fn)>(c);
  Py_RETURN_NONE;
}

// own_word(device, address): the library's status word of a device
PyObject *own_word(PyObject *, PyObject *args) {
  int dev;
  unsigned long long p;
  if (!PyArg_ParseTuple(args, "iK", &dev, &p)) return nullptr;
  if (dev >= 0 && dev < kMaxDevices) own_words[dev] = reinterpret_cast<int32_t *>(p);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(quantize_fp8, linear_fp8, cross_attention): addresses"},
    {"own_word", own_word, METH_VARARGS, "own_word(device, address)"},
    {"quantize_fp8", method(&guarded<quantize, 4>), METH_FASTCALL, "(x, rows, out, scale)"},
    {"linear_fp8", method(&guarded<linear, 10>), METH_FASTCALL,
     "(x, x_scale, w, w_scale, bias, act, gate, residual, out, status)"},
    {"cross_attention", method(&guarded<cross, 8>), METH_FASTCALL,
     "(q, k, v, lengths, mask, scale, out, status)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
