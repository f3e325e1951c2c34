// The common case of the linear layer's Python wrappers, in C++: contiguous
// operands, outputs made here, the current stream and device. In Python the
// checks, allocations and the marshalling take 5 to 7 us a call, longer than
// the smallest kernels and their launch; here 1 to 2. Whatever does not fit
// returns NotImplemented, before anything is enqueued, and the Python wrapper
// takes the call: it alone words the refusals.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

using at::ScalarType;
using at::Tensor;

struct Entry {
  int (*rmsnorm)(const void*, const void*, const void*, void*, float*, void*, int64_t, int64_t,
                 int64_t, int64_t, int64_t, int64_t, float, int, int, void*);
  int (*grad_bytes)(int64_t, int64_t, size_t*);
  int (*grad)(const void*, const void*, const void*, const void*, void*, float*, int64_t, int64_t,
              int64_t, int64_t, int64_t, int64_t, float, int, void*, size_t, void*);
  int (*fp8_bytes)(int64_t, int64_t, int64_t, size_t*);
  int (*fp8)(const void*, const float*, const void*, const float*, void*, int64_t, int64_t, int64_t,
             int64_t, int64_t, int64_t, int, void*, size_t, void*);
  int (*w4_bytes)(int64_t, int64_t, int64_t, size_t*);
  int (*w4)(const void*, const void*, const void*, const void*, void*, int64_t, int64_t, int64_t,
            int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, void*, size_t, void*);
  int (*layernorm)(const void*, const void*, const void*, const void*, void*, void*, void*, int64_t,
                   int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int, int, void*);
  int (*layer_grad_bytes)(int64_t, int64_t, size_t*);
  int (*layer_grad)(const void*, const void*, const void*, const void*, void*, float*, float*, int64_t,
                    int64_t, int64_t, int64_t, int64_t, int64_t, float, int, void*, size_t, void*);
  int (*quantize)(const void*, void*, void*, int64_t, int64_t, int64_t, int64_t, int64_t, int, void*);
  int (*dequantize)(const void*, const void*, void*, int64_t, int64_t, int64_t, int64_t, int64_t, int,
                    void*);
  int (*mx_bytes)(int64_t, int64_t, int64_t, size_t*);
  int (*mx)(const void*, const void*, const void*, const void*, void*, int64_t, int64_t, int64_t, int64_t,
            int64_t, int64_t, int64_t, int64_t, int, void*, size_t, void*);
};
Entry entry{};
PyObject* current_stream = nullptr;   // device -> address of its current stream

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

// A plain tensor or parameter; subclasses are the Python wrapper's.
const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// The address of an operand that may be missing. It throws for a tensor without
// storage (a function transform's), so it is read while the interpreter's lock
// is held, as every address here.
const void* address(const Tensor* t) { return t != nullptr ? t->const_data_ptr() : nullptr; }

int code16(ScalarType t) { return t == ScalarType::BFloat16 ? 0 : t == ScalarType::Half ? 1 : -1; }

bool matrix(const Tensor* t, ScalarType type, c10::Device dev, int64_t rows, int64_t cols) {
  return t != nullptr && t->scalar_type() == type && t->device() == dev && t->dim() == 2 &&
         t->size(0) == rows && t->size(1) == cols && t->is_contiguous();
}
bool vector(const Tensor* t, ScalarType type, c10::Device dev, int64_t n) {
  return t != nullptr && t->scalar_type() == type && t->device() == dev && t->dim() == 1 &&
         t->size(0) == n && t->is_contiguous();
}

// A plain 2-D operand on the current device, that is no subclass's, and the
// device's current stream.
bool begin(PyObject* o, const Tensor*& t, void*& stream) {
  if (!THPVariable_CheckExact(o)) return false;
  t = &THPVariable_Unpack(o);
  if (t->dim() != 2 || !t->is_cuda() || !t->is_contiguous()) return false;
  const c10::impl::VirtualGuardImpl guard(t->device().type());
  if (guard.getDevice() != t->device()) return false;
  PyObject* index = PyLong_FromLong(t->device().index());
  if (index == nullptr) return false;
  PyObject* raw = PyObject_CallOneArg(current_stream, index);
  Py_DECREF(index);
  if (raw == nullptr) return false;
  stream = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  return !PyErr_Occurred();
}

// An uninitialised tensor from the allocator that `like` came from: what at::empty
// ends in, without its way through the dispatcher (0.3 us).
Tensor make(const Tensor& like, c10::IntArrayRef size, ScalarType type) {
  c10::Allocator* allocator = like.storage().allocator();
  if (allocator == nullptr) return at::empty(size, like.options().dtype(type).requires_grad(false));
  return at::detail::empty_generic(size, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                   std::nullopt);
}

// The C call without the interpreter's lock, which is taken again however the
// call is left.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class... P, class... A>
int enqueue(int (*f)(P...), A... args) {
  const Unlocked unlocked;
  return f(args...);
}

PyObject* pack(std::initializer_list<const Tensor*> list) {
  PyObject* out = PyTuple_New((Py_ssize_t)list.size());
  if (out == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : list) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(*t));
  return out;
}

// rmsnorm(x, weight, residual or None, eps, out_dtype or None)
PyObject* rmsnorm(PyObject* const* a) {
  const Tensor* x;
  void* stream;
  if (!begin(a[0], x, stream)) return nullptr;
  const ScalarType type = x->scalar_type();
  const int code = code16(type);
  if (code < 0) return nullptr;
  ScalarType out = type;
  if (a[4] != Py_None) {
    if (!THPDtype_Check(a[4])) return nullptr;
    out = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
  }
  const bool q8 = out == ScalarType::Float8_e4m3fn;
  if (!q8 && out != type) return nullptr;
  const int64_t M = x->size(0), N = x->size(1);
  const Tensor *w = tensor(a[1]), *res = nullptr;
  if (!vector(w, type, x->device(), N)) return nullptr;
  if (a[2] != Py_None) {
    res = tensor(a[2]);
    if (!matrix(res, type, x->device(), M, N)) return nullptr;
  }
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const Tensor y = make(*x, {M, N}, out);
  Tensor s, h;
  if (q8) s = make(*x, {M}, ScalarType::Float);
  if (res != nullptr) h = make(*x, {M, N}, type);
  const int status = enqueue(entry.rmsnorm, address(x), address(res), address(w), y.data_ptr(),
                             q8 ? s.data_ptr<float>() : nullptr, res ? h.data_ptr() : nullptr, M, N, N,
                             N, N, N, (float)eps, code, q8 ? 3 : code, stream);
  if (status != 0) return nullptr;
  if (q8) return res ? pack({&y, &s, &h}) : pack({&y, &s});
  return res ? pack({&y, &h}) : THPVariable_Wrap(y);
}

// grad(dy, x, weight, dh or None, eps)
PyObject* grad(PyObject* const* a) {
  const Tensor* x;
  void* stream;
  if (!begin(a[1], x, stream)) return nullptr;
  const ScalarType type = x->scalar_type();
  const int code = code16(type);
  const int64_t M = x->size(0), N = x->size(1);
  const Tensor *dy = tensor(a[0]), *w = tensor(a[2]), *dh = nullptr;
  if (code < 0 || !matrix(dy, type, x->device(), M, N) || !vector(w, type, x->device(), N))
    return nullptr;
  if (a[3] != Py_None) {
    dh = tensor(a[3]);
    if (!matrix(dh, type, x->device(), M, N)) return nullptr;
  }
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  size_t bytes = 0;
  if (entry.grad_bytes(M, N, &bytes) != 0) return nullptr;
  const Tensor dx = make(*x, {M, N}, type), dw = make(*x, {N}, ScalarType::Float);
  Tensor ws;
  if (bytes > 0) ws = make(*x, {(int64_t)bytes}, ScalarType::Byte);
  const int status = enqueue(entry.grad, address(dy), address(x), address(w), address(dh), dx.data_ptr(),
                             dw.data_ptr<float>(), M, N, N, N, N, N, (float)eps, code,
                             bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
  return status != 0 ? nullptr : pack({&dx, &dw});
}

// gemm_fp8(A, a_scales, B, b_scales, out_dtype or None)
PyObject* gemm_fp8(PyObject* const* a) {
  constexpr ScalarType kE4 = ScalarType::Float8_e4m3fn;
  const Tensor* A;
  void* stream;
  if (!begin(a[0], A, stream)) return nullptr;
  const Tensor *sa = tensor(a[1]), *B = tensor(a[2]), *sb = tensor(a[3]);
  if (A->scalar_type() != kE4 || B == nullptr || B->scalar_type() != kE4 || B->dim() != 2 ||
      B->device() != A->device())
    return nullptr;
  const int64_t M = A->size(0), K = A->size(1), N = B->size(1);
  // B is the transpose of a contiguous N x K matrix.
  if (B->size(0) != K || K < 2 || N < 2 || B->stride(0) != 1 || B->stride(1) != K ||
      !vector(sa, ScalarType::Float, A->device(), M) || !vector(sb, ScalarType::Float, A->device(), N))
    return nullptr;
  ScalarType out = ScalarType::BFloat16;
  if (a[4] != Py_None) {
    if (!THPDtype_Check(a[4])) return nullptr;
    out = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
  }
  const int code = out == ScalarType::Float ? 2 : code16(out);
  size_t bytes = 0;
  if (code < 0 || entry.fp8_bytes(M, N, K, &bytes) != 0) return nullptr;
  const Tensor C = make(*A, {M, N}, out);
  Tensor ws;
  if (bytes > 0) ws = make(*A, {(int64_t)bytes}, ScalarType::Byte);
  const int status = enqueue(entry.fp8, address(A), static_cast<const float*>(address(sa)), address(B),
                             static_cast<const float*>(address(sb)), C.data_ptr(), M, N, K, K, K, N, code,
                             bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
  return status != 0 ? nullptr : THPVariable_Wrap(C);
}

// gemm_w4(A, codes, scales, zeros or None)
PyObject* gemm_w4(PyObject* const* a) {
  const Tensor* A;
  void* stream;
  if (!begin(a[0], A, stream)) return nullptr;
  const ScalarType type = A->scalar_type();
  const int code = code16(type);
  const Tensor *q = tensor(a[1]), *s = tensor(a[2]), *z = nullptr;
  const int64_t M = A->size(0), K = A->size(1);
  if (code < 0 || q == nullptr || q->dim() != 2 || s == nullptr || s->dim() != 2) return nullptr;
  const int64_t N = q->size(0), groups = s->size(1);
  if (K % 2 != 0 || groups <= 0 || K % groups != 0 ||
      !matrix(q, ScalarType::Byte, A->device(), N, K / 2) || !matrix(s, type, A->device(), N, groups))
    return nullptr;
  if (a[3] != Py_None) {
    z = tensor(a[3]);
    if (!matrix(z, ScalarType::Byte, A->device(), N, groups)) return nullptr;
  }
  size_t bytes = 0;
  if (entry.w4_bytes(M, N, K, &bytes) != 0) return nullptr;
  const Tensor C = make(*A, {M, N}, type);
  Tensor ws;
  if (bytes > 0) ws = make(*A, {(int64_t)bytes}, ScalarType::Byte);
  const int status = enqueue(entry.w4, address(A), address(q), address(s), address(z), C.data_ptr(), M, N, K,
                             K / groups, K, K / 2, groups, groups, N, code,
                             bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
  return status != 0 ? nullptr : THPVariable_Wrap(C);
}

// The 4-bit form's types; Undefined, which no tensor has, where torch lacks one.
template <class T, class = void>
struct Form {
  static constexpr T kF4 = T::Undefined, kE8 = T::Undefined;
};
template <class T>
struct Form<T, std::void_t<decltype(T::Float4_e2m1fn_x2), decltype(T::Float8_e8m0fnu)>> {
  static constexpr T kF4 = T::Float4_e2m1fn_x2, kE8 = T::Float8_e8m0fnu;
};
constexpr ScalarType kF4 = Form<ScalarType>::kF4, kE8 = Form<ScalarType>::kE8;

int code32(ScalarType t) { return t == ScalarType::Float ? 2 : code16(t); }

// The type that an argument names, `given` where it is None; no type where it is
// neither.
ScalarType dtype(PyObject* o, ScalarType given) {
  if (o == Py_None) return given;
  return THPDtype_Check(o) ? reinterpret_cast<THPDtype*>(o)->scalar_type : ScalarType::Undefined;
}

int64_t padded(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// e8m0 scales of rows that start at multiples of 16 bytes.
Tensor make_scales(const Tensor& like, int64_t rows, int64_t blocks) {
  const Tensor t = make(like, {rows, padded(blocks)}, kE8);
  const int64_t sizes[] = {rows, blocks}, strides[] = {padded(blocks), 1};
  t.unsafeGetTensorImpl()->set_sizes_and_strides(c10::IntArrayRef(sizes), c10::IntArrayRef(strides));
  return t;
}

// Their pitch, -1 for what the Python wrapper has to word. Rows are read in groups of
// 16 bytes, the last one too.
int64_t scales_pitch(const Tensor* t, c10::Device dev, int64_t rows, int64_t blocks) {
  if (t == nullptr || t->scalar_type() != kE8 || t->device() != dev || t->dim() != 2 ||
      t->size(0) != rows || t->size(1) != blocks || (blocks > 1 && t->stride(1) != 1))
    return -1;
  const int64_t pitch = rows > 1 ? t->stride(0) : padded(blocks);
  if (rows == 0 || pitch < blocks ||
      t->storage_offset() + (rows - 1) * pitch + padded(blocks) > (int64_t)t->storage().nbytes())
    return -1;
  return pitch;
}

// layernorm(x, weight, bias or None, residual or None, eps, out_dtype or None)
PyObject* layernorm(PyObject* const* a) {
  const Tensor* x;
  void* stream;
  if (!begin(a[0], x, stream)) return nullptr;
  const ScalarType type = x->scalar_type(), out = dtype(a[5], type);
  const int code = code16(type);
  const bool q8 = out == ScalarType::Float8_e4m3fn, mx = out == kF4;
  if (code < 0 || out == ScalarType::Undefined || (!q8 && !mx && out != type)) return nullptr;
  const int64_t M = x->size(0), N = x->size(1);
  if (mx && N % 32 != 0) return nullptr;
  const Tensor *w = tensor(a[1]), *b = nullptr, *res = nullptr;
  if (!vector(w, type, x->device(), N)) return nullptr;
  if (a[2] != Py_None) {
    b = tensor(a[2]);
    if (!vector(b, type, x->device(), N)) return nullptr;
  }
  if (a[3] != Py_None) {
    res = tensor(a[3]);
    if (!matrix(res, type, x->device(), M, N)) return nullptr;
  }
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int64_t columns = mx ? N / 2 : N, blocks = N / 32;
  const Tensor y = make(*x, {M, columns}, out);
  Tensor s, h;
  if (q8) s = make(*x, {M}, ScalarType::Float);
  if (mx) s = make_scales(*x, M, blocks);
  if (res != nullptr) h = make(*x, {M, N}, type);
  const int status = enqueue(entry.layernorm, address(x), address(res), address(w), address(b), y.data_ptr(),
                             q8 || mx ? s.data_ptr() : nullptr, res ? h.data_ptr() : nullptr, M, N, N, N,
                             columns, mx ? padded(blocks) : 0, N, (float)eps, code, mx ? 4 : q8 ? 3 : code,
                             stream);
  if (status != 0) return nullptr;
  if (q8 || mx) return res ? pack({&y, &s, &h}) : pack({&y, &s});
  return res ? pack({&y, &h}) : THPVariable_Wrap(y);
}

// layer_grad(dy, x, weight, dh or None, eps)
PyObject* layer_grad(PyObject* const* a) {
  const Tensor* x;
  void* stream;
  if (!begin(a[1], x, stream)) return nullptr;
  const ScalarType type = x->scalar_type();
  const int code = code16(type);
  const int64_t M = x->size(0), N = x->size(1);
  const Tensor *dy = tensor(a[0]), *w = tensor(a[2]), *dh = nullptr;
  if (code < 0 || !matrix(dy, type, x->device(), M, N) || !vector(w, type, x->device(), N))
    return nullptr;
  if (a[3] != Py_None) {
    dh = tensor(a[3]);
    if (!matrix(dh, type, x->device(), M, N)) return nullptr;
  }
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  size_t bytes = 0;
  if (entry.layer_grad_bytes(M, N, &bytes) != 0) return nullptr;
  const Tensor dx = make(*x, {M, N}, type), dw = make(*x, {N}, ScalarType::Float),
               db = make(*x, {N}, ScalarType::Float);
  Tensor ws;
  if (bytes > 0) ws = make(*x, {(int64_t)bytes}, ScalarType::Byte);
  const int status = enqueue(entry.layer_grad, address(dy), address(x), address(w), address(dh), dx.data_ptr(),
                             dw.data_ptr<float>(), db.data_ptr<float>(), M, N, N, N, N, N, (float)eps, code,
                             bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
  return status != 0 ? nullptr : pack({&dx, &dw, &db});
}

// quantize(x)
PyObject* quantize(PyObject* const* a) {
  const Tensor* x;
  void* stream;
  if (!begin(a[0], x, stream)) return nullptr;
  const int code = code32(x->scalar_type());
  const int64_t M = x->size(0), K = x->size(1);
  if (kF4 == ScalarType::Undefined || code < 0 || K % 32 != 0) return nullptr;
  const Tensor c = make(*x, {M, K / 2}, kF4), s = make_scales(*x, M, K / 32);
  const int status = enqueue(entry.quantize, address(x), c.data_ptr(), s.data_ptr(), M, K, K, K / 2,
                             padded(K / 32), code, stream);
  return status != 0 ? nullptr : pack({&c, &s});
}

// dequantize(codes, scales, out_dtype or None)
PyObject* dequantize(PyObject* const* a) {
  const Tensor* c;
  void* stream;
  if (!begin(a[0], c, stream) || c->scalar_type() != kF4) return nullptr;
  const ScalarType out = dtype(a[2], ScalarType::BFloat16);
  const int code = code32(out);
  const int64_t M = c->size(0), K = 2 * c->size(1);
  const Tensor* s = tensor(a[1]);
  if (code < 0 || K % 32 != 0) return nullptr;
  const int64_t ld_s = scales_pitch(s, c->device(), M, K / 32);
  if (ld_s < 0) return nullptr;
  const Tensor x = make(*c, {M, K}, out);
  const int status = enqueue(entry.dequantize, address(c), address(s), x.data_ptr(), M, K, K / 2, ld_s, K, code,
                             stream);
  return status != 0 ? nullptr : THPVariable_Wrap(x);
}

// gemm_mxfp4(A, a_scales, W, w_scales, out_dtype or None)
PyObject* gemm_mxfp4(PyObject* const* a) {
  const Tensor* A;
  void* stream;
  if (!begin(a[0], A, stream) || A->scalar_type() != kF4) return nullptr;
  const Tensor *sa = tensor(a[1]), *W = tensor(a[2]), *sw = tensor(a[3]);
  if (W == nullptr || W->dim() != 2) return nullptr;
  const int64_t M = A->size(0), bytes_row = A->size(1), K = 2 * bytes_row, N = W->size(0);
  if (K % 32 != 0 || !matrix(W, kF4, A->device(), N, bytes_row)) return nullptr;
  const int64_t ld_sa = scales_pitch(sa, A->device(), M, K / 32);
  const int64_t ld_sw = scales_pitch(sw, A->device(), N, K / 32);
  if (ld_sa < 0 || ld_sw < 0) return nullptr;
  const ScalarType out = dtype(a[4], ScalarType::BFloat16);
  const int code = code32(out);
  size_t bytes = 0;
  if (code < 0 || entry.mx_bytes(M, N, K, &bytes) != 0) return nullptr;
  const Tensor C = make(*A, {M, N}, out);
  Tensor ws;
  if (bytes > 0) ws = make(*A, {(int64_t)bytes}, ScalarType::Byte);
  const int status = enqueue(entry.mx, address(A), address(sa), address(W), address(sw), C.data_ptr(), M, N, K,
                             bytes_row, ld_sa, bytes_row, ld_sw, N, code, bytes > 0 ? ws.data_ptr() : nullptr,
                             bytes, stream);
  return status != 0 ? nullptr : THPVariable_Wrap(C);
}

// No exception leaves, and every failure (of an allocation too) is the Python
// wrapper's to meet again and report.
template <PyObject* (*F)(PyObject* const*), int N, bool LAYER = false>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != N || current_stream == nullptr || (LAYER && entry.layernorm == nullptr)) return not_here();
  PyObject* r = nullptr;
  try {
    r = F(args);
  } catch (const std::exception&) {
    r = nullptr;
  }
  if (r != nullptr) return r;
  PyErr_Clear();
  return not_here();
}

bool addresses(PyObject* const* args, void* (&at)[7]) {
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
      return false;
    }
  }
  return true;
}

// bind(current_stream, addresses of the seven entry points up to pipe_gemm_w4)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes a function and seven addresses");
    return nullptr;
  }
  void* at[7];
  if (!addresses(args + 1, at)) return nullptr;
  entry.rmsnorm = reinterpret_cast<decltype(entry.rmsnorm)>(at[0]);
  entry.grad_bytes = reinterpret_cast<decltype(entry.grad_bytes)>(at[1]);
  entry.grad = reinterpret_cast<decltype(entry.grad)>(at[2]);
  entry.fp8_bytes = reinterpret_cast<decltype(entry.fp8_bytes)>(at[3]);
  entry.fp8 = reinterpret_cast<decltype(entry.fp8)>(at[4]);
  entry.w4_bytes = reinterpret_cast<decltype(entry.w4_bytes)>(at[5]);
  entry.w4 = reinterpret_cast<decltype(entry.w4)>(at[6]);
  Py_INCREF(args[0]);
  Py_XDECREF(current_stream);
  current_stream = args[0];
  Py_RETURN_NONE;
}

// bind_layer(addresses of the seven entry points from pipe_layernorm on)
PyObject* bind_layer(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != 7) {
    PyErr_SetString(PyExc_TypeError, "bind_layer takes seven addresses");
    return nullptr;
  }
  void* at[7];
  if (!addresses(args, at)) return nullptr;
  entry.layer_grad_bytes = reinterpret_cast<decltype(entry.layer_grad_bytes)>(at[1]);
  entry.layer_grad = reinterpret_cast<decltype(entry.layer_grad)>(at[2]);
  entry.quantize = reinterpret_cast<decltype(entry.quantize)>(at[3]);
  entry.dequantize = reinterpret_cast<decltype(entry.dequantize)>(at[4]);
  entry.mx_bytes = reinterpret_cast<decltype(entry.mx_bytes)>(at[5]);
  entry.mx = reinterpret_cast<decltype(entry.mx)>(at[6]);
  entry.layernorm = reinterpret_cast<decltype(entry.layernorm)>(at[0]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"rmsnorm", FAST((guarded<rmsnorm, 5>)), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", FAST((guarded<grad, 5>)), METH_FASTCALL, nullptr},
    {"gemm_fp8", FAST((guarded<gemm_fp8, 5>)), METH_FASTCALL, nullptr},
    {"gemm_w4", FAST((guarded<gemm_w4, 4>)), METH_FASTCALL, nullptr},
    {"bind_layer", FAST(bind_layer), METH_FASTCALL, nullptr},
    {"layernorm", FAST((guarded<layernorm, 6, true>)), METH_FASTCALL, nullptr},
    {"layernorm_backward", FAST((guarded<layer_grad, 5, true>)), METH_FASTCALL, nullptr},
    {"quantize_mxfp4", FAST((guarded<quantize, 1, true>)), METH_FASTCALL, nullptr},
    {"dequantize_mxfp4", FAST((guarded<dequantize, 3, true>)), METH_FASTCALL, nullptr},
    {"gemm_mxfp4", FAST((guarded<gemm_mxfp4, 5, true>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_linear", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__linear(void) { return PyModule_Create(&module); }
