// Argument marshalling of the operators around the tail for Python: takes a tensor's type,
// shape, strides, device and address, checks what C cannot see in a bare pointer, and calls the
// C ABI.  The launch takes some 1.7 us on the host, as long as several of the kernels; a call
// through ctypes with checks in Python took 6 to 8 us, and reading the tensors by their Python
// attributes 0.3 us each (a norm of six tensors 4.2 us, now 2.1).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>

#include <cstdint>
#include <exception>

#include "../../include/klt.h"

namespace {

enum Kinds { BF16 = 1 << KLT_DT_BF16, F32 = 1 << KLT_DT_F32, CODES = 1 << KLT_DT_E4M3 };

struct Tensor {
  uint64_t ptr;
  int dtype;            // enum klt_dtype (codes: e4m3 or their bytes)
  long long size[2];    // rows, columns
  long long stride[2];  // elements
};

// Reads a tensor of one of `kinds` on `device` (< 0: any CUDA device, which it sets): a matrix,
// or with `broadcast` a row or a single number too.
bool read(PyObject* o, const char* name, int kinds, long long* device, Tensor* v,
          bool broadcast = false) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: not a tensor", name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  switch (t.scalar_type()) {
    case at::kBFloat16: v->dtype = KLT_DT_BF16; break;
    case at::kFloat: v->dtype = KLT_DT_F32; break;
    case at::kFloat8_e4m3fn:
    case at::kByte: v->dtype = KLT_DT_E4M3; break;
    default: v->dtype = 31;
  }
  if (!(kinds >> v->dtype & 1)) {
    PyErr_Format(PyExc_TypeError, "%s: dtype %s is not taken here", name,
                 c10::toString(t.scalar_type()));
    return false;
  }
  if (!t.is_cuda() || t.layout() != at::kStrided) {
    PyErr_Format(PyExc_ValueError, "%s: not a CUDA tensor with strides", name);
    return false;
  }
  const long long dev = t.get_device();
  if (*device < 0) *device = dev;
  if (dev != *device) {
    PyErr_Format(PyExc_ValueError, "%s: on CUDA device %lld, not %lld", name, dev, *device);
    return false;
  }
  const int64_t n = t.dim();
  if (n > 2 || (n != 2 && !broadcast)) {
    PyErr_Format(PyExc_ValueError, "%s: not a matrix", name);
    return false;
  }
  v->size[0] = v->size[1] = 1;
  v->stride[0] = v->stride[1] = 0;
  for (int64_t i = 0; i < n; ++i) {  // from the back: a vector is a row
    v->size[2 - n + i] = t.size(i);
    v->stride[2 - n + i] = t.stride(i);
  }
  v->ptr = reinterpret_cast<uintptr_t>(t.data_ptr());
  return true;
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

// `fn` with `device` current, on `stream` (None: torch's current one there); its status.  The
// interpreter's lock is free meanwhile: a launch waits where the stream's queue is full, and what
// has to run before it may be a host function that takes the lock.
template <typename Fn>
PyObject* launch(long long device, PyObject* stream, Fn fn) {
  void* s;
  if (stream == Py_None) {
    s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  } else {
    s = reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(stream)));
    if (PyErr_Occurred()) return nullptr;
  }
  int now = 0, rc = KLT_ERR_CUDA;
  Py_BEGIN_ALLOW_THREADS
  if (cudaGetDevice(&now) == cudaSuccess) {
    const bool other = now != device;
    if (!other || cudaSetDevice(static_cast<int>(device)) == cudaSuccess) rc = fn(s);
    if (other) cudaSetDevice(now);
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
  return false;
}
template <typename T>
T* address(const Tensor& v) {
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
    return klt_quantize(address<void>(x), x.dtype, x.stride[0], static_cast<int32_t>(M),
                        static_cast<int32_t>(K), address<uint8_t>(q), q.stride[0],
                        address<float>(s), stream);
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
  p.h = address<void>(t);
  p.h_dtype = t.dtype;
  p.ld_h = t.stride[0];
  const int stream_kind = 1 << t.dtype;
  if (a[3] != Py_None) {
    if (!read_rows(a[3], "y", BF16 | F32, &dev, M, H, false, &t)) return nullptr;
    p.y = address<void>(t);
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
    p.gate = address<void>(t);
    p.gate_dtype = t.dtype;
    p.gate_row = t.size[0] == 1 ? 0 : t.stride[0];
    p.gate_col = t.size[1] == 1 ? 0 : t.stride[1];
  }
  if (a[5] != Py_None) {
    if (!read_rows(a[5], "h_out", stream_kind, &dev, M, H, false, &t)) return nullptr;
    p.h_out = address<void>(t);
    p.ld_h_out = t.stride[0];
  }
  if (a[6] != Py_None) {
    if (!read_rows(a[6], "n", BF16, &dev, M, H, false, &t)) return nullptr;
    p.n = address<void>(t);
    p.ld_n = t.stride[0];
  }
  if (a[7] != Py_None) {
    if (!read_rows(a[7], "q", CODES, &dev, M, H, false, &t)) return nullptr;
    p.q = address<uint8_t>(t);
    p.ld_q = t.stride[0];
  }
  if (a[8] != Py_None) {
    if (!read_rows(a[8], "s", F32, &dev, M, (H + 127) / 128, true, &t)) return nullptr;
    p.s = address<float>(t);
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
    return klt_linear_forward(h, address<uint8_t>(xq), ld, address<float>(xs),
                              static_cast<int32_t>(M), address<void>(out), out.stride[0], address<float>(out_s),
                              static_cast<const klt_linear_debug*>(dbg), stream);
  });
}

// An entry point from which no C++ exception leaves (a tensor without memory throws one).
template <PyObject* (*FN)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return FN(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject* (*FN)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<FN>));
}
PyMethodDef methods[] = {{"quantize", entry<quantize>(), METH_FASTCALL, nullptr},
                         {"block_norm", entry<block_norm>(), METH_FASTCALL, nullptr},
                         {"linear", entry<linear>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
