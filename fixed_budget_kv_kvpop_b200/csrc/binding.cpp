// Argument marshalling of the paged cache's and kvpop_qk_norm_rope's calls for
// Python.  These are made once per layer and token, and the kernels behind the
// small ones run for 2 to 6 us; checking a tensor attribute by attribute from
// Python took 1 us, so the checks of a call (device, dtype, shape, strides,
// alignment, as include/kvpop.h asks) and the call itself are here.  No
// arithmetic of the operators is.  Each function takes the address of the C
// ABI call that it makes, so that any build of the library can stand behind it.
#include <Python.h>

#include <cmath>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/kvpop.h"

namespace {

// Arguments that every call has: where its tensors lie and what they hold.
struct Place {
  int device;
  at::ScalarType dtype;
};

bool refuse(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s: %s", name, what);
  return false;
}

bool tensor(PyObject* o, const char* name, const at::Tensor** out) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s: expected a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
    return false;
  }
  *out = &THPVariable_Unpack(o);
  return true;
}

bool refuse_shape(const char* name, const at::Tensor& t, at::IntArrayRef shape) {
  std::string got = "[", want = "[";
  for (const auto s : t.sizes()) got += std::to_string(s) + " ";
  for (const auto s : shape) want += std::to_string(s) + " ";
  PyErr_Format(PyExc_ValueError, "%s: shape %s], expected %s]", name, got.c_str(), want.c_str());
  return false;
}

// Device, dtype and shape.
bool fits(const at::Tensor& t, const char* name, const Place& at, at::ScalarType dtype, at::IntArrayRef shape) {
  if (!t.is_cuda() || t.get_device() != at.device) {
    PyErr_Format(PyExc_ValueError, "%s: on %s, expected the cuda device %d", name, t.device().str().c_str(), at.device);
    return false;
  }
  if (t.scalar_type() != dtype) {
    PyErr_Format(PyExc_ValueError, "%s: dtype %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(dtype));
    return false;
  }
  if (t.sizes() != shape) return refuse_shape(name, t, shape);
  return true;
}

// Rows [batch][token][head][head_dim], the last dimension contiguous, any strides of whole 16 bytes.
bool rows(PyObject* o, const char* name, const Place& at, at::IntArrayRef shape, bool written, kvpop_rows* out) {
  const at::Tensor* t;
  if (!tensor(o, name, &t) || !fits(*t, name, at, at.dtype, shape)) return false;
  const auto s = t->strides();
  const int64_t unit = at.dtype == at::kFloat ? 4 : 8;
  const bool empty = shape[0] == 0 || shape[1] == 0;
  void* p = t->data_ptr();
  bool odd = s[3] != 1 || (reinterpret_cast<uintptr_t>(p) & 15) != 0, wide = false;
  for (int i = 0; i < 3; ++i) {
    if (shape[i] <= 1) continue;
    odd |= s[i] % unit != 0;
    wide |= s[i] == 0;
  }
  if (odd && !empty)
    return refuse(name, "its strides or address are not whole 16 bytes, or its last dimension is not contiguous");
  if (written && wide && !empty) return refuse(name, "an expanded tensor cannot be written");
  *out = kvpop_rows{p, s[0], s[1], s[2]};
  return true;
}

bool dense(PyObject* o, const char* name, const Place& at, at::ScalarType dtype, at::IntArrayRef shape, void** out) {
  const at::Tensor* t;
  if (!tensor(o, name, &t) || !fits(*t, name, at, dtype, shape)) return false;
  if (!t->is_contiguous()) return refuse(name, "must be contiguous");
  *out = t->data_ptr();
  return true;
}

bool ints(PyObject* o, const char* name, const Place& at, at::IntArrayRef shape, const int32_t** out) {
  void* p;
  if (!dense(o, name, at, at::kInt, shape, &p)) return false;
  *out = static_cast<const int32_t*>(p);
  return true;
}

// The first two dimensions of rows that set the size of a call.
bool batch_of(PyObject* o, const char* name, int64_t* b, int64_t* n) {
  const at::Tensor* t;
  if (!tensor(o, name, &t)) return false;
  if (t->dim() != 4) return refuse(name, "expected a cuda tensor [batch][tokens][heads][head_dim]");
  *b = t->size(0);
  *n = t->size(1);
  if (*b > INT32_MAX || *n > INT32_MAX) return refuse(name, "too many rows");
  return true;
}

bool whole(PyObject* o, int64_t* out) {
  *out = PyLong_AsLongLong(o);
  return *out != -1 || !PyErr_Occurred();
}
bool whole32(PyObject* o, const char* name, int32_t* out) {
  int64_t v;
  if (!whole(o, &v)) return false;
  if (v < INT32_MIN || v > INT32_MAX) return refuse(name, "does not fit 32 bits");
  *out = static_cast<int32_t>(v);
  return true;
}
template <typename F>
bool pointer(PyObject* o, F** out) {
  *out = reinterpret_cast<F*>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

// The stream given (a torch stream), or the device's current one, which need not be the current device's.
bool stream_of(PyObject* o, int device, void** out) {
  if (o == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    return true;
  }
  PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
  if (!s) return false;
  const bool ok = pointer(s, out);
  Py_DECREF(s);
  return ok;
}

// A tuple (handle, q heads, KV heads, head_dim, dtype code, device) that a cache keeps.
struct Cache {
  kvpop_paged_handle* h;
  int32_t hq, hkv, d;
  Place at;
};
bool cache_of(PyObject* o, Cache* c) {
  int32_t code, device;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) return refuse("cache", "expected its tuple of six");
  if (!pointer(PyTuple_GET_ITEM(o, 0), &c->h) || !whole32(PyTuple_GET_ITEM(o, 1), "heads", &c->hq) ||
      !whole32(PyTuple_GET_ITEM(o, 2), "heads", &c->hkv) || !whole32(PyTuple_GET_ITEM(o, 3), "head_dim", &c->d) ||
      !whole32(PyTuple_GET_ITEM(o, 4), "dtype", &code) || !whole32(PyTuple_GET_ITEM(o, 5), "device", &device))
    return false;
  c->at = Place{device, code == KVPOP_DTYPE_F32 ? at::kFloat : at::kBFloat16};
  return true;
}

// A tuple (packed kvpop_rope, device, head_dim or 0) that a Rope keeps.
bool rope_of(PyObject* o, int device, int64_t d, const kvpop_rope** out) {
  int32_t dev, dim;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3 || !PyBytes_Check(PyTuple_GET_ITEM(o, 0)) ||
      PyBytes_GET_SIZE(PyTuple_GET_ITEM(o, 0)) != static_cast<Py_ssize_t>(sizeof(kvpop_rope)))
    return refuse("rope", "expected a Rope (make_rope)");
  if (!whole32(PyTuple_GET_ITEM(o, 1), "rope", &dev) || !whole32(PyTuple_GET_ITEM(o, 2), "rope", &dim)) return false;
  if (dev != device) return refuse("rope", "on another device than the rows");
  if (dim != 0 && dim != d) return refuse("rope", "its weights are not head_dim elements long");
  *out = reinterpret_cast<const kvpop_rope*>(PyBytes_AS_STRING(PyTuple_GET_ITEM(o, 0)));
  return true;
}

bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return false;
}

template <typename F>
PyObject* call(F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

// qk_norm_rope(fn, rope, q, k, positions, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  decltype(kvpop_qk_norm_rope)* fn;
  int64_t b, t, b2, t2;
  if (!counted(n, 8) || !pointer(a[0], &fn) || !batch_of(a[2], "q", &b, &t) || !batch_of(a[3], "k", &b2, &t2)) return nullptr;
  const at::Tensor &q = THPVariable_Unpack(a[2]), &k = THPVariable_Unpack(a[3]);
  const int64_t hq = q.size(2), hkv = k.size(2), d = q.size(3);
  if (!q.is_cuda()) { refuse("q", "expected a cuda tensor"); return nullptr; }
  if (q.scalar_type() != at::kFloat && q.scalar_type() != at::kBFloat16) { refuse("q", "dtype: expected float32 or bfloat16"); return nullptr; }
  if (hq > INT32_MAX || hkv > INT32_MAX || d > INT32_MAX) { refuse("q", "too many heads"); return nullptr; }
  const Place at{q.get_device(), q.scalar_type()};
  const kvpop_rope* rope;
  kvpop_rows qr, kr, qo, ko;
  const int32_t* pos;
  void* st;
  if (!rope_of(a[1], at.device, d, &rope) || !rows(a[2], "q", at, {b, t, hq, d}, false, &qr) ||
      !rows(a[3], "k", at, {b, t, hkv, d}, false, &kr) || !ints(a[4], "positions", at, {b, t}, &pos) ||
      !rows(a[5], "q_out", at, {b, t, hq, d}, true, &qo) || !rows(a[6], "k_out", at, {b, t, hkv, d}, true, &ko) ||
      !stream_of(a[7], at.device, &st))
    return nullptr;
  const int code = at.dtype == at::kFloat ? KVPOP_DTYPE_F32 : KVPOP_DTYPE_BF16;
  return call([&] {
    return fn(code, static_cast<int32_t>(d), static_cast<int32_t>(hq), static_cast<int32_t>(hkv), rope,
              static_cast<int32_t>(b), static_cast<int32_t>(t), &qr, &kr, pos, &qo, &ko, st);
  });
}

// append(fn, cache, layer, k, v, slots, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  decltype(kvpop_paged_append)* fn;
  Cache c;
  int32_t layer;
  int64_t b, t;
  kvpop_rows k, v;
  const int32_t* slots;
  void* st;
  if (!counted(n, 7) || !pointer(a[0], &fn) || !cache_of(a[1], &c) || !whole32(a[2], "layer", &layer) ||
      !batch_of(a[3], "k", &b, &t) || !rows(a[3], "k", c.at, {b, t, c.hkv, c.d}, false, &k) ||
      !rows(a[4], "v", c.at, {b, t, c.hkv, c.d}, false, &v) || !ints(a[5], "slots", c.at, {b, t}, &slots) ||
      !stream_of(a[6], c.at.device, &st))
    return nullptr;
  return call([&] { return fn(c.h, layer, &k, &v, slots, static_cast<int32_t>(b), static_cast<int32_t>(t), st); });
}

// append_qkv(fn, cache, layer, rope, q, k, v, positions, slots, q_out, stream)
PyObject* append_qkv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  decltype(kvpop_paged_append_qkv)* fn;
  Cache c;
  int32_t layer;
  int64_t b, t;
  const kvpop_rope* rope;
  kvpop_rows q, k, v, qo;
  const int32_t *pos, *slots;
  void* st;
  if (!counted(n, 11) || !pointer(a[0], &fn) || !cache_of(a[1], &c) || !whole32(a[2], "layer", &layer) ||
      !rope_of(a[3], c.at.device, c.d, &rope) || !batch_of(a[5], "k", &b, &t) ||
      !rows(a[4], "q", c.at, {b, t, c.hq, c.d}, false, &q) || !rows(a[5], "k", c.at, {b, t, c.hkv, c.d}, false, &k) ||
      !rows(a[6], "v", c.at, {b, t, c.hkv, c.d}, false, &v) || !ints(a[7], "positions", c.at, {b, t}, &pos) ||
      !ints(a[8], "slots", c.at, {b, t}, &slots) || !rows(a[9], "q_out", c.at, {b, t, c.hq, c.d}, true, &qo) ||
      !stream_of(a[10], c.at.device, &st))
    return nullptr;
  return call([&] {
    return fn(c.h, layer, rope, &q, &k, &v, pos, slots, &qo, static_cast<int32_t>(b), static_cast<int32_t>(t), st);
  });
}

// Page table [batch][pages] and lengths [batch].
bool tables(PyObject* table, PyObject* lens, const Place& at, int64_t b, const int32_t** tp, int32_t* width, const int32_t** lp) {
  const at::Tensor* t;
  if (!tensor(table, "page_table", &t)) return false;
  if (t->dim() != 2) return refuse("page_table", "expected an int32 cuda tensor [batch][pages]");
  const int64_t w = t->size(1);
  if (w > INT32_MAX) return refuse("page_table", "too wide");
  *width = static_cast<int32_t>(w);
  return ints(table, "page_table", at, {b, w}, tp) && ints(lens, "lens", at, {b}, lp);
}

// gather(fn, cache, layer, page_table, lens, k_out, v_out, stream)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  decltype(kvpop_paged_gather)* fn;
  Cache c;
  int32_t layer, width;
  int64_t b, t;
  kvpop_rows k, v;
  const int32_t *table, *lens;
  void* st;
  if (!counted(n, 8) || !pointer(a[0], &fn) || !cache_of(a[1], &c) || !whole32(a[2], "layer", &layer) ||
      !batch_of(a[5], "k_out", &b, &t) || !tables(a[3], a[4], c.at, b, &table, &width, &lens) ||
      !rows(a[5], "k_out", c.at, {b, t, c.hkv, c.d}, true, &k) ||
      !rows(a[6], "v_out", c.at, {b, t, c.hkv, c.d}, true, &v) || !stream_of(a[7], c.at.device, &st))
    return nullptr;
  return call([&] {
    return fn(c.h, layer, table, width, width, lens, static_cast<int32_t>(b), static_cast<int32_t>(t), &k, &v, st);
  });
}

// attend(fn, cache, layer, q, page_table, lens, out, lse, scale, softcap, window, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  decltype(kvpop_paged_attend)* fn;
  Cache c;
  int32_t layer, width;
  const at::Tensor* qt;
  const int32_t *table, *lens;
  void *q, *out, *lse = nullptr, *st;
  kvpop_attend_options o;
  if (!counted(n, 12) || !pointer(a[0], &fn) || !cache_of(a[1], &c) || !whole32(a[2], "layer", &layer) || !tensor(a[3], "q", &qt))
    return nullptr;
  if (qt->dim() != 3 || qt->size(0) > INT32_MAX) { refuse("q", "expected a cuda tensor [batch][q heads][head_dim]"); return nullptr; }
  const int64_t b = qt->size(0);
  if (!dense(a[3], "q", c.at, c.at.dtype, {b, c.hq, c.d}, &q) || !dense(a[6], "out", c.at, c.at.dtype, {b, c.hq, c.d}, &out) ||
      (a[7] != Py_None && !dense(a[7], "lse", c.at, at::kFloat, {b, c.hq}, &lse)) ||
      !tables(a[4], a[5], c.at, b, &table, &width, &lens) || !whole32(a[10], "window", &o.window) ||
      !stream_of(a[11], c.at.device, &st))
    return nullptr;
  const double scale = PyFloat_AsDouble(a[8]), cap = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred()) return nullptr;
  // 0 is the default: what only rounds to 0 is not taken for it
  o.scale = scale != 0 && static_cast<float>(scale) == 0.f ? NAN : static_cast<float>(scale);
  o.softcap = cap != 0 && static_cast<float>(cap) == 0.f ? NAN : static_cast<float>(cap);
  return call([&] {
    return fn(c.h, layer, q, table, width, width, lens, static_cast<int32_t>(b), &o, out, static_cast<float*>(lse), st);
  });
}

// Nothing that a call throws (torch's own errors) leaves it as a C++ exception.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction method() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)); }

PyMethodDef methods[] = {
    {"qk_norm_rope", method<qk_norm_rope>(), METH_FASTCALL, nullptr},
    {"append", method<append>(), METH_FASTCALL, nullptr},
    {"append_qkv", method<append_qkv>(), METH_FASTCALL, nullptr},
    {"gather", method<gather>(), METH_FASTCALL, nullptr},
    {"attend", method<attend>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Tells the loader which torch and Python it was compiled for.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddStringConstant(m, "TORCH", TORCH_VERSION) < 0 || PyModule_AddIntConstant(m, "PYTHON", PY_VERSION_HEX >> 16) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
