// The 8-bit calls' Python side (module _binding): checks of the tensors' types,
// shapes, layouts and devices, the outputs' allocation through torch.empty, and
// the call of the C ABI on the current stream.  Marshalling only, as in
// __init__.py, but a decode step makes these calls by the hundred and the same
// checks written in Python cost 4 us of a 9 us call.  Needs Python's headers,
// not torch's: tensors are asked through their Python methods.
//
// Every function returns NotImplemented when its tensors are on another device
// than the current one; __init__.py then makes that device current and calls
// again.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "../../include/paro.h"

namespace {

// Interned names and what the module keeps of torch.
PyObject *n_dtype, *n_shape, *n_device, *n_get_device, *n_is_contiguous, *n_data_ptr;
PyObject *t_int8, *t_f32, *t_bf16, *t_f16, *t_int16, *t_uint16, *t_uint8;
PyObject *f_empty, *f_empty_like, *f_stream, *f_device, *k_empty, *f_check;

// The C ABI's entry points, as the library that __init__.py loaded has them.
struct Api {
  decltype(&paro_quantize_activations_int8) quantize;
  decltype(&paro_rms_norm_int8) norm;
  decltype(&paro_pack_weights_int8) pack;
  decltype(&paro_w8a8_linear) linear;
  decltype(&paro_w8a8_swiglu) swiglu;
  decltype(&paro_rotate_w8a8_workspace_bytes) rotate_bytes;
  decltype(&paro_rotate_w8a8_linear) rotate;
} api;

// A reference that is given back at the end of its scope.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o = nullptr) : p(o) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

bool given(PyObject* o) { return o != Py_None; }

PyObject* method(PyObject* t, PyObject* name) {
  return PyObject_VectorcallMethod(name, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, nullptr);
}

// A two-dimensional tensor's sizes.
bool rows_of(PyObject* t, const char* name, long long (&d)[2]) {
  Ref s(PyObject_GetAttr(t, n_shape));
  if (!s.p) return false;
  if (!PyTuple_Check(s.p) || PyTuple_GET_SIZE(s.p) != 2) {
    PyErr_Format(PyExc_ValueError, "%s must have two dimensions, got %R", name, s.p);
    return false;
  }
  for (int i = 0; i < 2; ++i) d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s.p, i));
  if (PyErr_Occurred()) return false;
  if (d[0] > INT32_MAX || d[1] > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s: %R is beyond 2^31 - 1 rows or columns", name, s.p);
    return false;
  }
  return true;
}

bool device_of(PyObject* t, int* dev) {
  Ref d(method(t, n_get_device));
  if (!d.p) return false;
  *dev = (int)PyLong_AsLong(d.p);
  return !PyErr_Occurred();
}

// The tensor's address, after checks; sizes of -1 are not checked.  None: null.
bool address(PyObject* t, PyObject* dtype, int n, const long long* sizes, int dev, const char* name, void** out) {
  *out = nullptr;
  if (!given(t)) return true;
  Ref ty(PyObject_GetAttr(t, n_dtype)), s(PyObject_GetAttr(t, n_shape));
  if (!ty.p || !s.p) return false;
  bool same = ty.p == dtype && PyTuple_Check(s.p) && PyTuple_GET_SIZE(s.p) == n;
  for (int i = 0; same && i < n; ++i) same = PyLong_AsLongLong(PyTuple_GET_ITEM(s.p, i)) == sizes[i];
  if (PyErr_Occurred()) return false;
  if (!same) {
    Ref want(PyTuple_New(n));
    for (int i = 0; want.p && i < n; ++i) PyTuple_SET_ITEM(want.p, i, PyLong_FromLongLong(sizes[i]));
    PyErr_Format(PyExc_ValueError, "%s: expected %R %R, got %R %R", name, dtype, want.p, ty.p, s.p);
    return false;
  }
  int at = -1;
  if (!device_of(t, &at)) return false;
  if (at < 0 || at != dev) {
    PyErr_Format(PyExc_ValueError, "%s: expected a tensor of the same CUDA device as the first one", name);
    return false;
  }
  Ref c(method(t, n_is_contiguous));
  if (!c.p) return false;
  if (c.p != Py_True) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor", name);
    return false;
  }
  Ref a(method(t, n_data_ptr));
  if (!a.p) return false;
  *out = PyLong_AsVoidPtr(a.p);
  return !PyErr_Occurred();
}

// bf16 or fp16 as the C ABI numbers them.
bool act_type(PyObject* dtype, paro_dtype* out) {
  if (dtype == t_bf16) *out = PARO_BF16;
  else if (dtype == t_f16) *out = PARO_FP16;
  else {
    PyErr_Format(PyExc_ValueError, "expected bfloat16 or float16, got %R", dtype);
    return false;
  }
  return true;
}

// A first tensor's device, if that is current (1), else 0; -1 on error.
int current(int dev) {
  if (dev < 0) return 1;  // a CPU tensor: refused by its check
  Ref d(PyObject_CallNoArgs(f_device));
  if (!d.p) return -1;
  const long at = PyLong_AsLong(d.p);
  return PyErr_Occurred() ? -1 : at == dev;
}

bool stream_of(int dev, paro_stream_t* out) {
  Ref n(PyLong_FromLong(dev));
  if (!n.p) return false;
  Ref s(PyObject_CallOneArg(f_stream, n.p));
  if (!s.p) return false;
  *out = (paro_stream_t)PyLong_AsVoidPtr(s.p);
  return !PyErr_Occurred();
}

// A new tensor (or null after an error) with its address in *out.
PyObject* addressed(PyObject* made, void** out) {
  if (!made) return nullptr;
  Ref p(method(made, n_data_ptr));
  if (!p.p) {
    Py_DECREF(made);
    return nullptr;
  }
  *out = PyLong_AsVoidPtr(p.p);
  return made;
}

// `t` itself after its check, or a new tensor beside `like`; its address to *out.
PyObject* output(PyObject* t, PyObject* dtype, int n, const long long* sizes, int dev, PyObject* like, const char* name,
                 void** out) {
  if (given(t)) {
    if (!address(t, dtype, n, sizes, dev, name, out)) return nullptr;
    Py_INCREF(t);
    return t;
  }
  Ref d(PyObject_GetAttr(like, n_device)), a(PyLong_FromLongLong(sizes[0])), b(n > 1 ? PyLong_FromLongLong(sizes[1]) : nullptr);
  if (!d.p || !a.p || (n > 1 && !b.p)) return nullptr;
  PyObject* args[4];
  int k = 0;
  args[k++] = a.p;
  if (n > 1) args[k++] = b.p;
  args[k] = dtype;
  args[k + 1] = d.p;
  return addressed(PyObject_Vectorcall(f_empty, args, k, k_empty), out);
}

// Calls the library, with the interpreter's lock given up (a launch may wait for
// room in the stream's queue), and raises ParoError for a status that is not OK.
template <typename F, typename... A>
bool run(const char* what, F fn, A... args) {
  paro_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(args...);
  Py_END_ALLOW_THREADS
  if (st == PARO_OK) return true;
  Ref r(PyObject_CallFunction(f_check, "is", (int)st, what));
  if (r.p) PyErr_SetString(PyExc_RuntimeError, what);
  return false;
}

bool count(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
  return false;
}

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

// quantize(x, q, sx) -> (q, sx)
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 3, "quantize")) return nullptr;
  long long d[2];
  int dev, here;
  paro_dtype ty;
  void *x, *q, *sx;
  paro_stream_t s;
  if (!rows_of(v[0], "x", d) || !device_of(v[0], &dev) || (here = current(dev)) < 0) return nullptr;
  if (!here) return not_here();
  Ref t(PyObject_GetAttr(v[0], n_dtype));
  if (!t.p || !act_type(t.p, &ty) || !address(v[0], t.p, 2, d, dev, "x", &x)) return nullptr;
  Ref oq(output(v[1], t_int8, 2, d, dev, v[0], "q", &q));
  if (!oq.p) return nullptr;
  Ref os(output(v[2], t_f32, 1, d, dev, v[0], "sx", &sx));
  if (!os.p || !stream_of(dev, &s)) return nullptr;
  if (!run("paro_quantize_activations_int8", api.quantize, (uint16_t*)x, (int8_t*)q, (float*)sx, (int)d[0], (int)d[1], ty, s))
    return nullptr;
  return PyTuple_Pack(2, oq.p, os.p);
}

// norm(x, gain, residual, eps, hidden, q, sx) -> (q, sx, hidden)
PyObject* norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 7, "norm")) return nullptr;
  long long d[2];
  int dev, here;
  paro_dtype ty;
  void *x, *g, *r, *h = nullptr, *q, *sx;
  paro_stream_t s;
  if (!given(v[2]) && given(v[4])) {
    PyErr_SetString(PyExc_ValueError, "hidden is written only with a residual");
    return nullptr;
  }
  if (!rows_of(v[0], "x", d) || !device_of(v[0], &dev) || (here = current(dev)) < 0) return nullptr;
  if (!here) return not_here();
  const double eps = PyFloat_AsDouble(v[3]);
  if (PyErr_Occurred()) return nullptr;
  Ref t(PyObject_GetAttr(v[0], n_dtype));
  if (!t.p || !act_type(t.p, &ty) || !address(v[0], t.p, 2, d, dev, "x", &x) ||
      !address(v[2], t.p, 2, d, dev, "residual", &r) || !address(v[1], t.p, 1, d + 1, dev, "gain", &g))
    return nullptr;
  Ref oh(!given(v[2])  ? Py_NewRef(Py_None)
         : given(v[4]) ? output(v[4], t.p, 2, d, dev, v[0], "hidden", &h)
                       : addressed(PyObject_CallOneArg(f_empty_like, v[0]), &h));
  if (!oh.p) return nullptr;
  Ref oq(output(v[5], t_int8, 2, d, dev, v[0], "q", &q));
  if (!oq.p) return nullptr;
  Ref os(output(v[6], t_f32, 1, d, dev, v[0], "sx", &sx));
  if (!os.p || !stream_of(dev, &s)) return nullptr;
  if (!run("paro_rms_norm_int8", api.norm, (uint16_t*)x, (uint16_t*)r, (uint16_t*)g, (float)eps, (uint16_t*)h, (int8_t*)q,
           (float*)sx, (int)d[0], (int)d[1], ty, s))
    return nullptr;
  return PyTuple_Pack(3, oq.p, os.p, oh.p);
}

// A transform's tables for width d: pairs (v[0]), cos_t, sin_t, scale.
struct Tables {
  long long K = 0;
  void *pairs = nullptr, *cos = nullptr, *sin = nullptr, *scale = nullptr;
  bool take(PyObject* const* v, long long d, int dev) {
    if (!address(v[3], t_f32, 1, &d, dev, "scale", &scale)) return false;
    if (!given(v[0])) return true;
    Ref shape(PyObject_GetAttr(v[0], n_shape)), t(PyObject_GetAttr(v[0], n_dtype));
    if (!shape.p || !t.p) return false;
    K = PyTuple_Check(shape.p) && PyTuple_GET_SIZE(shape.p) == 3 ? PyLong_AsLongLong(PyTuple_GET_ITEM(shape.p, 0)) : -1;
    if (PyErr_Occurred()) return false;
    if (K < 0 || K > 1 << 20 || (t.p != t_int16 && t.p != t_uint16) || !given(v[1]) || !given(v[2])) {
      PyErr_SetString(PyExc_ValueError, "a transform takes int16 or uint16 pairs [K, d/2, 2], cos_t and sin_t");
      return false;
    }
    const long long sizes[3] = {K, d / 2, 2};
    return address(v[0], t.p, 3, sizes, dev, "pairs", &pairs) && address(v[1], t_f32, 2, sizes, dev, "cos_t", &cos) &&
           address(v[2], t_f32, 2, sizes, dev, "sin_t", &sin);
  }
};

// pack(W, pairs, cos_t, sin_t, scale, workspace, qweight, wscales) -> (qweight, wscales)
PyObject* pack(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 8, "pack")) return nullptr;
  long long d[2];
  int dev, here;
  Tables t;
  void *W, *ws = nullptr, *q, *ss;
  paro_stream_t s;
  if (!rows_of(v[0], "W", d) || !device_of(v[0], &dev) || (here = current(dev)) < 0) return nullptr;
  if (!here) return not_here();
  if (!address(v[0], t_f32, 2, d, dev, "W", &W) || !t.take(v + 1, d[1], dev)) return nullptr;
  Ref ow(t.K > 0 || t.scale ? output(v[5], t_f32, 2, d, dev, v[0], "workspace", &ws) : Py_NewRef(Py_None));
  if (!ow.p) return nullptr;
  Ref oq(output(v[6], t_int8, 2, d, dev, v[0], "qweight", &q));
  if (!oq.p) return nullptr;
  Ref os(output(v[7], t_f32, 1, d, dev, v[0], "wscales", &ss));
  if (!os.p || !stream_of(dev, &s)) return nullptr;
  if (!run("paro_pack_weights_int8", api.pack, (float*)W, (int)d[0], (int)d[1], (int)t.K, (uint16_t*)t.pairs, (float*)t.cos,
           (float*)t.sin, (float*)t.scale, (float*)ws, (int8_t*)q, (float*)ss, s))
    return nullptr;
  return PyTuple_Pack(2, oq.p, os.p);
}

// linear(q, sx, qweight, wscales, bias, out, out_dtype) -> out, and with GATED
// swiglu(q, sx, gate_qweight, gate_wscales, up_qweight, up_wscales, out, out_dtype) -> out
template <bool GATED>
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
  constexpr int O = GATED ? 6 : 5;
  if (!count(n, O + 2, GATED ? "swiglu" : "linear")) return nullptr;
  long long a[2], b[2];
  int dev, here;
  paro_dtype ty;
  void *q, *sx, *w, *sw, *w2 = nullptr, *s2 = nullptr, *bias = nullptr, *y;
  paro_stream_t s;
  if (!rows_of(v[0], "q", a) || !rows_of(v[2], GATED ? "gate_qweight" : "qweight", b) || !device_of(v[0], &dev) ||
      (here = current(dev)) < 0)
    return nullptr;
  if (!here) return not_here();
  Ref t(given(v[O]) ? PyObject_GetAttr(v[O], n_dtype) : Py_NewRef(v[O + 1]));
  if (!t.p || !act_type(t.p, &ty)) return nullptr;
  const long long wsize[2] = {b[0], a[1]}, ysize[2] = {a[0], b[0]};
  if (!address(v[0], t_int8, 2, a, dev, "q", &q) || !address(v[1], t_f32, 1, a, dev, "sx", &sx) ||
      !address(v[2], t_int8, 2, wsize, dev, GATED ? "gate_qweight" : "qweight", &w) ||
      !address(v[3], t_f32, 1, wsize, dev, GATED ? "gate_wscales" : "wscales", &sw))
    return nullptr;
  if (GATED) {
    if (!address(v[4], t_int8, 2, wsize, dev, "up_qweight", &w2) || !address(v[5], t_f32, 1, wsize, dev, "up_wscales", &s2))
      return nullptr;
  } else if (!address(v[4], t.p, 1, wsize, dev, "bias", &bias)) {
    return nullptr;
  }
  Ref oy(output(v[O], t.p, 2, ysize, dev, v[0], "out", &y));
  if (!oy.p || !stream_of(dev, &s)) return nullptr;
  const int M = (int)a[0], d_in = (int)a[1], d_out = (int)b[0];
  if (!(GATED ? run("paro_w8a8_swiglu", api.swiglu, (int8_t*)q, (float*)sx, (int8_t*)w, (float*)sw, (int8_t*)w2, (float*)s2,
                    (uint16_t*)y, M, d_in, d_out, ty, s)
              : run("paro_w8a8_linear", api.linear, (int8_t*)q, (float*)sx, (int8_t*)w, (float*)sw, (uint16_t*)bias,
                    (uint16_t*)y, M, d_in, d_out, ty, s)))
    return nullptr;
  return Py_NewRef(oy.p);
}

// rotate_linear(x, pairs, cos_t, sin_t, scale, qweight, wscales, bias, out, workspace) -> out
PyObject* rotate_linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 10, "rotate_linear")) return nullptr;
  long long a[2], b[2];
  int dev, here;
  Tables t;
  void *x, *w, *sw, *bias, *y, *ws;
  paro_stream_t s;
  if (!rows_of(v[0], "x", a) || !rows_of(v[5], "qweight", b) || !device_of(v[0], &dev) || (here = current(dev)) < 0)
    return nullptr;
  if (!here) return not_here();
  const long long wsize[2] = {b[0], a[1]}, ysize[2] = {a[0], b[0]};
  if (!address(v[0], t_bf16, 2, a, dev, "x", &x) || !t.take(v + 1, a[1], dev) ||
      !address(v[5], t_int8, 2, wsize, dev, "qweight", &w) || !address(v[6], t_f32, 1, wsize, dev, "wscales", &sw) ||
      !address(v[7], t_bf16, 1, wsize, dev, "bias", &bias))
    return nullptr;
  Ref oy(output(v[8], t_bf16, 2, ysize, dev, v[0], "out", &y));
  if (!oy.p) return nullptr;
  long long bytes = (long long)api.rotate_bytes((int)a[0], (int)a[1]);
  if (given(v[9])) {
    Ref len(PyObject_GetAttr(v[9], n_shape));
    if (!len.p) return nullptr;
    bytes = PyTuple_Check(len.p) && PyTuple_GET_SIZE(len.p) == 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(len.p, 0)) : 0;
    if (PyErr_Occurred()) return nullptr;
  }
  Ref ow(output(v[9], t_uint8, 1, &bytes, dev, v[0], "workspace", &ws));
  if (!ow.p || !stream_of(dev, &s)) return nullptr;
  if (!run("paro_rotate_w8a8_linear", api.rotate, (uint16_t*)x, (int)t.K, (uint16_t*)t.pairs, (float*)t.cos, (float*)t.sin,
           (float*)t.scale, (int8_t*)w, (float*)sw, (uint16_t*)bias, (uint16_t*)y, (int)a[0], (int)a[1], (int)b[0], ws,
           (size_t)bytes, s))
    return nullptr;
  return Py_NewRef(oy.p);
}

// setup(torch, check, addresses): what the calls need of torch, what raises
// ParoError, and the C ABI's addresses in Api's order.
PyObject* setup(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 3, "setup")) return nullptr;
  auto get = [&](PyObject* from, const char* name, PyObject** to) {
    *to = from ? PyObject_GetAttrString(from, name) : nullptr;
    return *to != nullptr;
  };
  Ref c(PyObject_GetAttrString(v[0], "_C"));
  if (!c.p || !get(v[0], "int8", &t_int8) || !get(v[0], "float32", &t_f32) || !get(v[0], "bfloat16", &t_bf16) ||
      !get(v[0], "float16", &t_f16) || !get(v[0], "int16", &t_int16) || !get(v[0], "uint16", &t_uint16) ||
      !get(v[0], "uint8", &t_uint8) ||
      !get(v[0], "empty", &f_empty) ||
      !get(v[0], "empty_like", &f_empty_like) || !get(c.p, "_cuda_getCurrentRawStream", &f_stream) ||
      !get(c.p, "_cuda_getDevice", &f_device))
    return nullptr;
  f_check = Py_NewRef(v[1]);
  void** slots[] = {(void**)&api.quantize, (void**)&api.norm, (void**)&api.pack, (void**)&api.linear,
                    (void**)&api.swiglu, (void**)&api.rotate_bytes, (void**)&api.rotate};
  constexpr int kCalls = sizeof(slots) / sizeof(slots[0]);
  if (!PyTuple_Check(v[2]) || PyTuple_GET_SIZE(v[2]) != kCalls) {
    PyErr_SetString(PyExc_TypeError, "an address for each call is wanted");
    return nullptr;
  }
  for (int i = 0; i < kCalls; ++i)
    if (!(*slots[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(v[2], i)))) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, nullptr},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, nullptr},
    {"pack", (PyCFunction)(void (*)(void))pack, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void (*)(void))linear<false>, METH_FASTCALL, nullptr},
    {"swiglu", (PyCFunction)(void (*)(void))linear<true>, METH_FASTCALL, nullptr},
    {"rotate_linear", (PyCFunction)(void (*)(void))rotate_linear, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  n_dtype = PyUnicode_InternFromString("dtype");
  n_shape = PyUnicode_InternFromString("shape");
  n_device = PyUnicode_InternFromString("device");
  n_get_device = PyUnicode_InternFromString("get_device");
  n_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  k_empty = Py_BuildValue("(ss)", "dtype", "device");
  if (!n_dtype || !n_shape || !n_device || !n_get_device || !n_is_contiguous || !n_data_ptr || !k_empty) return nullptr;
  return PyModule_Create(&module);
}
