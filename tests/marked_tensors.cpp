// Host tensors that carry a device's mark, for tests without a device: the
// storage comes from an allocator of malloc, and so do tensors made from it.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/core/impl/FakeGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdlib>
#include <cstring>

namespace {

struct HostAllocator final : c10::Allocator {
  c10::DataPtr allocate(size_t n) override {
    void* p = n ? std::malloc(n) : nullptr;
    return {p, p, &std::free, c10::Device(c10::DeviceType::CUDA, 0)};
  }
  c10::DeleterFnPtr raw_deleter() const override { return &std::free; }
  void copy_data(void* to, const void* from, size_t n) const override { std::memcpy(to, from, n); }
};
HostAllocator allocator;
const c10::impl::FakeGuardImpl<c10::DeviceType::CUDA> device;   // current device 0, no runtime behind it

PyObject* marked(PyObject*, PyObject* o) {
  const at::Tensor& t = THPVariable_Unpack(o);
  return THPVariable_Wrap(at::detail::empty_generic(t.sizes(), &allocator,
                                                    c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                    t.scalar_type(), std::nullopt));
}
PyMethodDef methods[] = {{"marked", marked, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "marked_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_marked_tensors(void) {
  c10::impl::device_guard_impl_registry[(int)c10::DeviceType::CUDA].store(&device);
  return PyModule_Create(&module);
}
