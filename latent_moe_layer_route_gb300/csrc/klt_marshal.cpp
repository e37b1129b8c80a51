// Argument marshalling of the operators around the tail for Python: takes a tensor's type,
// shape, strides, device and address by the attributes that Python would read, checks what C
// cannot see in a bare pointer, and calls the C ABI.  A call through ctypes and checks in
// Python took 6 to 8 us on the host, as long as several of the kernels; this takes about half,
// most of it the launch itself.  No torch headers: the tensors are plain Python objects.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <cuda_runtime_api.h>

#include <cstdint>

#include "../../include/klt.h"

namespace {

// Attribute names and torch's objects, looked up on the first call.
PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr;
PyObject *t_bf16, *t_f32, *t_e4m3, *t_uint8, *t_stream;

bool load_torch() {
  if (t_stream) return true;
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return false;
  t_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  t_f32 = PyObject_GetAttrString(torch, "float32");
  t_e4m3 = PyObject_GetAttrString(torch, "float8_e4m3fn");
  t_uint8 = PyObject_GetAttrString(torch, "uint8");
  PyObject* c = PyObject_GetAttrString(torch, "_C");
  Py_DECREF(torch);
  if (!c) return false;
  PyObject* stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  if (!t_bf16 || !t_f32 || !t_e4m3 || !t_uint8 || !stream) return false;
  t_stream = stream;
  return true;
}

PyObject* call0(PyObject* self, PyObject* name) {
  PyObject* args[1] = {self};
  return PyObject_VectorcallMethod(name, args, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, nullptr);
}

// An integer result of a call, taken over; false with an exception set if it is none.
bool take_int(PyObject* v, long long* out) {
  if (!v) return false;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return *out != -1 || !PyErr_Occurred();
}

// A tuple of at most 2 integers, taken over, from the back (a vector is a row); n = its length.
bool take_pair(PyObject* v, Py_ssize_t* n, long long out[2]) {
  if (!v) return false;
  *n = PyTuple_Check(v) ? PyTuple_GET_SIZE(v) : -1;
  for (Py_ssize_t i = 0; *n <= 2 && i < *n; ++i) {
    out[2 - *n + i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    if (out[2 - *n + i] == -1 && PyErr_Occurred()) {
      Py_DECREF(v);
      return false;
    }
  }
  Py_DECREF(v);
  return true;
}

enum Kinds { BF16 = 1 << KLT_DT_BF16, F32 = 1 << KLT_DT_F32, CODES = 1 << KLT_DT_E4M3 };

struct Tensor {
  uint64_t ptr;
  int dtype;            // enum klt_dtype (codes: e4m3 or their bytes)
  long long size[2];    // rows, columns
  long long stride[2];  // elements
};

// Reads a tensor of one of `kinds` on `device` (< 0: any CUDA device, which it sets).
bool read(PyObject* t, const char* name, int kinds, long long* device, Tensor* v,
          bool broadcast = false) {
  PyObject* dtype = PyObject_GetAttr(t, s_dtype);
  if (!dtype) return false;
  v->dtype = dtype == t_bf16 ? KLT_DT_BF16
             : dtype == t_f32 ? KLT_DT_F32
             : dtype == t_e4m3 || dtype == t_uint8 ? KLT_DT_E4M3
                                                    : 31;
  const bool known = kinds >> v->dtype & 1;
  if (!known)
    PyErr_Format(PyExc_TypeError, "%s: dtype %R is not taken here", name, dtype);
  Py_DECREF(dtype);
  if (!known) return false;
  long long dev;
  if (!take_int(call0(t, s_get_device), &dev)) return false;
  if (dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s: not a CUDA tensor", name);
    return false;
  }
  if (*device < 0) *device = dev;
  if (dev != *device) {
    PyErr_Format(PyExc_ValueError, "%s: on CUDA device %lld, not %lld", name, dev, *device);
    return false;
  }
  Py_ssize_t n, m;
  v->size[0] = v->size[1] = 1;
  v->stride[0] = v->stride[1] = 0;
  if (!take_pair(PyObject_GetAttr(t, s_shape), &n, v->size) ||
      !take_pair(call0(t, s_stride), &m, v->stride))
    return false;
  if (n != m || n < 0 || n > 2 || (n != 2 && !broadcast)) {
    PyErr_Format(PyExc_ValueError, "%s: not a matrix", name);
    return false;
  }
  PyObject* ptr = call0(t, s_data_ptr);
  if (!ptr) return false;
  v->ptr = PyLong_AsUnsignedLongLong(ptr);
  Py_DECREF(ptr);
  return !PyErr_Occurred();
}

// ... of [rows, cols], its columns contiguous, the rows too if `whole`.
bool read_rows(PyObject* t, const char* name, int kinds, long long* device, long long rows,
               long long cols, bool whole, Tensor* v) {
  if (!read(t, name, kinds, device, v)) return false;
  if (v->size[0] != rows || v->size[1] != cols) {
    PyErr_Format(PyExc_ValueError, "%s: shape (%lld, %lld), not (%lld, %lld)", name, v->size[0],
                 v->size[1], rows, cols);
    return false;
  }
  if ((v->stride[1] != 1 && cols > 1) || (whole && v->stride[0] != cols && rows > 1)) {
    PyErr_Format(PyExc_ValueError, "%s: %s not contiguous", name, whole ? "" : "columns are");
    return false;
  }
  return true;
}

// `fn` with `device` current, on `stream` (None: torch's current one there); its status.
template <typename Fn>
PyObject* launch(long long device, PyObject* stream, Fn fn) {
  long long s;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLongLong(device);
    if (!d) return nullptr;
    PyObject* args[2] = {nullptr, d};
    PyObject* r =
        PyObject_Vectorcall(t_stream, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, nullptr);
    Py_DECREF(d);
    if (!take_int(r, &s)) return nullptr;
  } else {
    s = static_cast<long long>(PyLong_AsUnsignedLongLong(stream));
    if (PyErr_Occurred()) return nullptr;
  }
  int now = 0;
  if (cudaGetDevice(&now) != cudaSuccess) return PyLong_FromLong(KLT_ERR_CUDA);
  const bool other = now != device;
  if (other && cudaSetDevice(static_cast<int>(device)) != cudaSuccess)
    return PyLong_FromLong(KLT_ERR_CUDA);
  const int rc = fn(reinterpret_cast<void*>(static_cast<uintptr_t>(s)));
  if (other) cudaSetDevice(now);
  return PyLong_FromLong(rc);
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
    return false;
  }
  return load_torch();
}
template <typename T>
T* at(const Tensor& v) {
  return reinterpret_cast<T*>(static_cast<uintptr_t>(v.ptr));
}
bool as_int(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}
bool fits32(long long v, const char* name) {
  if (v <= INT32_MAX) return true;
  PyErr_Format(PyExc_ValueError, "%s: more than 2^31 - 1 rows or columns", name);
  return false;
}

// quantize(x, q, s, stream) -> status
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  long long dev = -1;
  Tensor x, q, s;
  if (!read(a[0], "x", BF16 | F32, &dev, &x)) return nullptr;
  const long long M = x.size[0], K = x.size[1];
  if (!fits32(M, "x") || !fits32(K, "x")) return nullptr;
  if (x.stride[1] != 1 && K > 1) {
    PyErr_SetString(PyExc_ValueError, "x: columns are not contiguous");
    return nullptr;
  }
  if (!read_rows(a[1], "q", CODES, &dev, M, K, false, &q) ||
      !read_rows(a[2], "s", F32, &dev, M, (K + 127) / 128, true, &s))
    return nullptr;
  return launch(dev, a[3], [&](void* stream) {
    return klt_quantize(at<void>(x), x.dtype, x.stride[0], static_cast<int32_t>(M),
                        static_cast<int32_t>(K), at<uint8_t>(q), q.stride[0], at<float>(s),
                        stream);
  });
}

// block_norm(address of the layer's klt_block_norm_args, device or -1, h, y, gate, h_out, n, q,
// s, stream) -> status; tensors may be None
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  const void* layer = PyLong_AsVoidPtr(a[0]);
  long long dev;
  if (!layer || !as_int(a[1], &dev)) return nullptr;
  klt_block_norm_args p = *static_cast<const klt_block_norm_args*>(layer);
  const long long H = p.H;
  Tensor t;
  if (!read(a[2], "h", BF16 | F32, &dev, &t)) return nullptr;
  const long long M = t.size[0];
  if (!fits32(M, "h")) return nullptr;
  if (t.size[1] != H || (t.stride[1] != 1 && H > 1)) {
    PyErr_Format(PyExc_ValueError, "h: not [rows, %lld] with contiguous columns", H);
    return nullptr;
  }
  p.M = static_cast<int32_t>(M);
  p.h = at<void>(t);
  p.h_dtype = t.dtype;
  p.ld_h = t.stride[0];
  const int stream_kind = 1 << t.dtype;
  if (a[3] != Py_None) {
    if (!read_rows(a[3], "y", BF16 | F32, &dev, M, H, false, &t)) return nullptr;
    p.y = at<void>(t);
    p.y_dtype = t.dtype;
    p.ld_y = t.stride[0];
  } else {
    p.gamma_post = nullptr;
  }
  if (a[4] != Py_None) {
    if (!p.y && M > 0) {
      PyErr_SetString(PyExc_ValueError, "gate: given without y");
      return nullptr;
    }
    if (!read(a[4], "gate", BF16 | F32, &dev, &t, true)) return nullptr;
    if ((t.size[0] != 1 && t.size[0] != M) || (t.size[1] != 1 && t.size[1] != H)) {
      PyErr_Format(PyExc_ValueError, "gate: (%lld, %lld) does not broadcast to (%lld, %lld)",
                   t.size[0], t.size[1], M, H);
      return nullptr;
    }
    p.gate = at<void>(t);
    p.gate_dtype = t.dtype;
    p.gate_row = t.size[0] == 1 ? 0 : t.stride[0];
    p.gate_col = t.size[1] == 1 ? 0 : t.stride[1];
  }
  if (a[5] != Py_None) {
    if (!read_rows(a[5], "h_out", stream_kind, &dev, M, H, false, &t)) return nullptr;
    p.h_out = at<void>(t);
    p.ld_h_out = t.stride[0];
  }
  if (a[6] != Py_None) {
    if (!read_rows(a[6], "n", BF16, &dev, M, H, false, &t)) return nullptr;
    p.n = at<void>(t);
    p.ld_n = t.stride[0];
  }
  if (a[7] != Py_None) {
    if (!read_rows(a[7], "q", CODES, &dev, M, H, false, &t)) return nullptr;
    p.q = at<uint8_t>(t);
    p.ld_q = t.stride[0];
  }
  if (a[8] != Py_None) {
    if (!read_rows(a[8], "s", F32, &dev, M, (H + 127) / 128, true, &t)) return nullptr;
    p.s = at<float>(t);
  }
  return launch(dev, a[9], [&](void* stream) { return klt_block_norm(&p, stream); });
}

// linear(handle, device, K, outputs, klt_dtype of the output, xq, xs, out, out_s, address of a
// klt_linear_debug or 0, stream) -> status
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  klt_linear* h = static_cast<klt_linear*>(PyLong_AsVoidPtr(a[0]));
  const void* dbg = PyLong_AsVoidPtr(a[9]);
  long long dev, K, width, dtype;
  if (PyErr_Occurred() || !as_int(a[1], &dev) || !as_int(a[2], &K) || !as_int(a[3], &width) ||
      !as_int(a[4], &dtype))
    return nullptr;
  Tensor xq, xs, out, out_s = {};
  if (!read(a[5], "xq", CODES, &dev, &xq)) return nullptr;
  const long long M = xq.size[0];
  if (!fits32(M, "xq")) return nullptr;
  if (xq.size[1] != K || (xq.stride[1] != 1 && K > 1)) {
    PyErr_Format(PyExc_ValueError, "xq: not [rows, %lld] with contiguous columns", K);
    return nullptr;
  }
  if (!read_rows(a[6], "xs", F32, &dev, M, (K + 127) / 128, true, &xs) ||
      !read_rows(a[7], "out", 1 << dtype, &dev, M, width, false, &out) ||
      (dtype == KLT_DT_E4M3 &&
       !read_rows(a[8], "out_s", F32, &dev, M, width / 128, true, &out_s)))
    return nullptr;
  // the stride of a single row says nothing
  const long long ld = M <= 1 ? (K + 15) / 16 * 16 : xq.stride[0];
  return launch(dev, a[10], [&](void* stream) {
    return klt_linear_forward(h, at<uint8_t>(xq), ld, at<float>(xs), static_cast<int32_t>(M),
                              at<void>(out), out.stride[0], at<float>(out_s),
                              static_cast<const klt_linear_debug*>(dbg), stream);
  });
}

PyMethodDef methods[] = {
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(quantize)), METH_FASTCALL,
     nullptr},
    {"block_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_norm)),
     METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_shape || !s_stride || !s_get_device || !s_data_ptr) return nullptr;
  return PyModule_Create(&module);
}
