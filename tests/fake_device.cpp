// Devices that are none, for tests of which device is current during a call of
// the binding: tensors on them (their memory is never touched), and a device
// guard that tells the stand-in for the CUDA runtime (fake_cudart.c).
#include <Python.h>

#include <ATen/ops/from_blob.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

extern "C" void fake_device(int);

namespace {

constexpr auto kType = c10::DeviceType::PrivateUse1;
int current = 0;

struct Guard final : c10::impl::DeviceGuardImplInterface {
  c10::DeviceType type() const override { return kType; }
  c10::Device getDevice() const override { return c10::Device(kType, (c10::DeviceIndex)current); }
  void uncheckedSetDevice(c10::Device d) const noexcept override { fake_device(current = d.index()); }
  void setDevice(c10::Device d) const override { uncheckedSetDevice(d); }
  c10::Device exchangeDevice(c10::Device d) const override {
    const c10::Device was = getDevice();
    setDevice(d);
    return was;
  }
  c10::Stream getStream(c10::Device d) const override { return c10::Stream(c10::Stream::DEFAULT, d); }
  c10::Stream exchangeStream(c10::Stream s) const override { return s; }
  c10::DeviceIndex deviceCount() const noexcept override { return 2; }
};
const Guard guard;
const c10::impl::DeviceGuardImplRegistrar registrar(kType, &guard);

// (device, like): a tensor of the shape, strides and type of `like` on that device
PyObject *tensor(PyObject *, PyObject *args) {
  int index;
  PyObject *o;
  if (!PyArg_ParseTuple(args, "iO", &index, &o)) return nullptr;
  const at::Tensor &like = THPVariable_Unpack(o);
  const c10::Device device(kType, (c10::DeviceIndex)index);
  return THPVariable_Wrap(at::for_blob(reinterpret_cast<void *>(1 << 20), like.sizes())
                              .strides(like.strides())
                              .options(like.options().device(device))
                              .target_device(device)
                              .make_tensor());
}
PyObject *now(PyObject *, PyObject *) { return PyLong_FromLong(current); }

PyMethodDef methods[] = {{"tensor", tensor, METH_VARARGS, nullptr}, {"current", now, METH_NOARGS, nullptr}, {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fake_device", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fake_device(void) { return PyModule_Create(&module); }
