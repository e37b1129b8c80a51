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

// A tensor of latent attention: its type, device and sizes are checked (a size < 0: any, which it
// sets), its last direction is contiguous; the strides of the others.
struct Strided {
  void* ptr = nullptr;
  int64_t size[3] = {1, 1, 1};
  int64_t stride[3] = {};
};
bool read_nd(PyObject* o, const char* name, at::ScalarType type, at::ScalarType other,
             long long device, int dims, const int64_t* want, Strided* v, bool whole = false) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: not a tensor", name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type && t.scalar_type() != other) {
    PyErr_Format(PyExc_TypeError, "%s: dtype %s is not taken here", name,
                 c10::toString(t.scalar_type()));
    return false;
  }
  if (!t.is_cuda() || t.layout() != at::kStrided) {
    PyErr_Format(PyExc_ValueError, "%s: not a CUDA tensor with strides", name);
    return false;
  }
  if (t.get_device() != device) {
    PyErr_Format(PyExc_ValueError, "%s: on CUDA device %lld, not %lld", name,
                 static_cast<long long>(t.get_device()), device);
    return false;
  }
  if (t.dim() != dims) {
    PyErr_Format(PyExc_ValueError, "%s: %lld dimensions, not %d", name,
                 static_cast<long long>(t.dim()), dims);
    return false;
  }
  for (int i = 0; i < dims; ++i) {
    v->size[i] = t.size(i);
    v->stride[i] = t.stride(i);
    if ((want[i] >= 0 && v->size[i] != want[i]) || v->size[i] > INT32_MAX) {
      PyErr_Format(PyExc_ValueError, "%s: size %lld in dimension %d, not %lld", name,
                   static_cast<long long>(v->size[i]), i,
                   static_cast<long long>(want[i] >= 0 ? want[i] : INT32_MAX));
      return false;
    }
  }
  if ((v->stride[dims - 1] != 1 && v->size[dims - 1] > 1) || (whole && !t.is_contiguous())) {
    PyErr_Format(PyExc_ValueError, "%s: not contiguous", name);
    return false;
  }
  v->ptr = t.data_ptr();
  return true;
}
bool read_nd(PyObject* o, const char* name, at::ScalarType type, long long device, int dims,
             const int64_t (&want)[3], Strided* v, bool whole = false) {
  return read_nd(o, name, type, type, device, dims, want, v, whole);
}
struct Latent {
  klt_latent* h;
  const klt_latent_dims* d;
  long long dev;
};
bool read_latent(PyObject* const* a, Latent* l) {
  l->h = static_cast<klt_latent*>(PyLong_AsVoidPtr(a[0]));
  l->d = static_cast<const klt_latent_dims*>(PyLong_AsVoidPtr(a[1]));
  return !PyErr_Occurred() && as_int(a[2], &l->dev);
}

// latent_append(handle, address of its klt_latent_dims, device, kv, positions, slots, cache, kv_out,
// q, q_out, stream) -> status; slots to q_out may be None
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Latent l;
  if (!arity(n, 11) || !read_latent(a, &l)) return nullptr;
  const int64_t width = l.d->latent + l.d->rope, H = l.d->heads;
  klt_latent_append_args p = {};
  Strided t;
  const int64_t kv_size[2] = {-1, width};
  if (!read_nd(a[3], "kv", at::kBFloat16, at::kFloat, l.dev, 2, kv_size, &t))
    return nullptr;
  const int64_t T = t.size[0];
  p.T = static_cast<int32_t>(T);
  p.kv = t.ptr;
  p.ld_kv = t.stride[0];
  p.kv_dtype =
      THPVariable_Unpack(a[3]).scalar_type() == at::kFloat ? KLT_DT_F32 : KLT_DT_BF16;
  if (T <= 1) p.ld_kv = 0;  // the stride of a single row says nothing
  if (!read_nd(a[4], "positions", at::kLong, l.dev, 1, {T}, &t, true)) return nullptr;
  p.positions = static_cast<const int64_t*>(t.ptr);
  if (a[5] != Py_None) {
    if (!read_nd(a[5], "slots", at::kLong, l.dev, 1, {T}, &t, true)) return nullptr;
    p.slots = static_cast<const int64_t*>(t.ptr);
  }
  if (a[6] != Py_None) {
    if (!read_nd(a[6], "cache", at::kBFloat16, l.dev, 3, {-1, l.d->page, width}, &t))
      return nullptr;
    p.cache = t.ptr;
    p.pages = t.size[0];
    p.page_stride = p.pages > 1 ? t.stride[0] : 0;
    p.row_stride = t.stride[1];
  }
  if (a[7] != Py_None) {
    if (!read_nd(a[7], "kv_out", at::kBFloat16, l.dev, 2, {T, width}, &t)) return nullptr;
    p.kv_out = t.ptr;
    p.ld_kv_out = T > 1 ? t.stride[0] : 0;
  }
  if (a[8] != Py_None) {
    if (!read_nd(a[8], "q", at::kBFloat16, l.dev, 3, {T, H, l.d->rope}, &t)) return nullptr;
    p.q = t.ptr;
    p.q_token = T > 1 ? t.stride[0] : 0;
    p.q_head = H > 1 ? t.stride[1] : 0;
  }
  if (a[9] != Py_None) {
    if (!read_nd(a[9], "q_out", at::kBFloat16, l.dev, 3, {T, H, l.d->rope}, &t)) return nullptr;
    p.q_out = t.ptr;
    p.q_out_token = T > 1 ? t.stride[0] : 0;
    p.q_out_head = H > 1 ? t.stride[1] : 0;
  }
  return launch(l.dev, a[10], [&](void* s) { return klt_latent_append(l.h, &p, s); });
}

// latent_attend(handle, dims, device, q, cache, block_table, seq_lens, cu_q or None, out, lse,
// workspace, address of a klt_latent_debug or 0, stream) -> status
PyObject* latent_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Latent l;
  if (!arity(n, 13) || !read_latent(a, &l)) return nullptr;
  const int64_t width = l.d->latent + l.d->rope, H = l.d->heads;
  const auto* dbg = static_cast<const klt_latent_debug*>(PyLong_AsVoidPtr(a[11]));
  if (PyErr_Occurred()) return nullptr;
  klt_latent_attend_args p = {};
  Strided t;
  if (!read_nd(a[3], "q", at::kBFloat16, l.dev, 3, {-1, H, width}, &t)) return nullptr;
  const int64_t T = t.size[0];
  p.T = static_cast<int32_t>(T);
  p.q = t.ptr;
  p.q_token = T > 1 ? t.stride[0] : 0;
  p.q_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[4], "cache", at::kBFloat16, l.dev, 3, {-1, l.d->page, width}, &t)) return nullptr;
  p.cache = t.ptr;
  p.pages = t.size[0];
  p.page_stride = p.pages > 1 ? t.stride[0] : 0;
  p.row_stride = t.stride[1];
  if (!read_nd(a[5], "block_table", at::kInt, l.dev, 2, {-1, -1}, &t)) return nullptr;
  const int64_t B = t.size[0];
  p.B = static_cast<int32_t>(B);
  p.max_pages = static_cast<int32_t>(t.size[1]);
  p.block_table = static_cast<const int32_t*>(t.ptr);
  p.ld_table = B > 1 ? t.stride[0] : 0;
  if (!read_nd(a[6], "seq_lens", at::kInt, l.dev, 1, {B}, &t, true)) return nullptr;
  p.seq_lens = static_cast<const int32_t*>(t.ptr);
  if (a[7] != Py_None) {
    if (!read_nd(a[7], "cu_q", at::kInt, l.dev, 1, {B + 1}, &t, true)) return nullptr;
    p.cu_q = static_cast<const int32_t*>(t.ptr);
  }
  if (!read_nd(a[8], "out", at::kBFloat16, l.dev, 3, {T, H, l.d->latent}, &t)) return nullptr;
  p.out = t.ptr;
  p.out_token = T > 1 ? t.stride[0] : 0;
  p.out_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[9], "lse", at::kFloat, l.dev, 2, {T, H}, &t, true)) return nullptr;
  p.lse = static_cast<float*>(t.ptr);
  if (!read_nd(a[10], "workspace", at::kByte, l.dev, 1, {-1}, &t, true)) return nullptr;
  p.workspace = t.ptr;
  p.workspace_bytes = static_cast<uint64_t>(t.size[0]);
  return launch(l.dev, a[12], [&](void* s) { return klt_latent_attend(l.h, &p, dbg, s); });
}

// latent_prefill(handle, dims, device, q, k, v, k_rope, cu_q, cu_k, causal, out, lse, address of a
// klt_latent_debug or 0, stream) -> status
PyObject* latent_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Latent l;
  if (!arity(n, 14) || !read_latent(a, &l)) return nullptr;
  const int64_t H = l.d->heads;
  const auto* dbg = static_cast<const klt_latent_debug*>(PyLong_AsVoidPtr(a[12]));
  if (PyErr_Occurred()) return nullptr;
  klt_latent_prefill_args p = {};
  Strided t;
  if (!read_nd(a[3], "q", at::kBFloat16, l.dev, 3, {-1, H, l.d->nope + l.d->rope}, &t))
    return nullptr;
  const int64_t T = t.size[0];
  p.T = static_cast<int32_t>(T);
  p.q = t.ptr;
  p.q_token = T > 1 ? t.stride[0] : 0;
  p.q_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[4], "k", at::kBFloat16, l.dev, 3, {-1, H, l.d->nope}, &t)) return nullptr;
  const int64_t S = t.size[0];
  p.S = static_cast<int32_t>(S);
  p.k = t.ptr;
  p.k_token = S > 1 ? t.stride[0] : 0;
  p.k_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[5], "v", at::kBFloat16, l.dev, 3, {S, H, l.d->value}, &t)) return nullptr;
  p.v = t.ptr;
  p.v_token = S > 1 ? t.stride[0] : 0;
  p.v_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[6], "k_rope", at::kBFloat16, l.dev, 2, {S, l.d->rope}, &t)) return nullptr;
  p.k_rope = t.ptr;
  p.ld_k_rope = S > 1 ? t.stride[0] : 0;
  if (!read_nd(a[7], "cu_q", at::kInt, l.dev, 1, {-1}, &t, true)) return nullptr;
  const int64_t starts = t.size[0];
  p.cu_q = static_cast<const int32_t*>(t.ptr);
  p.B = static_cast<int32_t>(starts - 1);
  if (!read_nd(a[8], "cu_k", at::kInt, l.dev, 1, {starts}, &t, true)) return nullptr;
  p.cu_k = static_cast<const int32_t*>(t.ptr);
  p.causal = PyObject_IsTrue(a[9]);
  if (!read_nd(a[10], "out", at::kBFloat16, l.dev, 3, {T, H, l.d->value}, &t)) return nullptr;
  p.out = t.ptr;
  p.out_token = T > 1 ? t.stride[0] : 0;
  p.out_head = H > 1 ? t.stride[1] : 0;
  if (!read_nd(a[11], "lse", at::kFloat, l.dev, 2, {T, H}, &t, true)) return nullptr;
  p.lse = static_cast<float*>(t.ptr);
  return launch(l.dev, a[13], [&](void* s) { return klt_latent_prefill(l.h, &p, dbg, s); });
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
                         {"latent_append", entry<latent_append>(), METH_FASTCALL, nullptr},
                         {"latent_attend", entry<latent_attend>(), METH_FASTCALL, nullptr},
                         {"latent_prefill", entry<latent_prefill>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
