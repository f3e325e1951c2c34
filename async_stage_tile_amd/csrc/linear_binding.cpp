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

// No exception leaves, and every failure (of an allocation too) is the Python
// wrapper's to meet again and report.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != N || current_stream == nullptr) return not_here();
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

// bind(current_stream, addresses of the seven entry points)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes a function and seven addresses");
    return nullptr;
  }
  void* at[7];
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
      return nullptr;
    }
  }
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

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"rmsnorm", FAST((guarded<rmsnorm, 5>)), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", FAST((guarded<grad, 5>)), METH_FASTCALL, nullptr},
    {"gemm_fp8", FAST((guarded<gemm_fp8, 5>)), METH_FASTCALL, nullptr},
    {"gemm_w4", FAST((guarded<gemm_w4, 4>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_linear", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__linear(void) { return PyModule_Create(&module); }
