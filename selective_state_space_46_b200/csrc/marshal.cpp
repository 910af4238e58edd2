// Writes a call's tensor descriptors for the Python binding.  A decode step is a few microseconds on the GPU;
// reading eight tensors' pointers, shapes and strides from Python takes longer than that.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "mssm.h"

namespace {

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MSSM_F32;
    case at::kBFloat16: return MSSM_BF16;
    case at::kInt: return MSSM_I32;
    case at::kByte: return MSSM_U8;
    default: return -1;
  }
}

// describe(block, *tensors) -> (device index, addresses): the descriptor of tensor j goes to block[j], and None
// stays None.  All tensors have to be on one CUDA device.
PyObject* describe(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 2) {
    PyErr_SetString(PyExc_TypeError, "describe(block, *tensors)");
    return nullptr;
  }
  auto* block = static_cast<mssm_tensor*>(PyLong_AsVoidPtr(args[0]));
  if (!block) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null descriptor block");
    return nullptr;
  }
  int device = -1;
  PyObject* out = PyTuple_New(n);
  if (!out) return nullptr;
  for (Py_ssize_t j = 1; j < n; ++j) {
    if (args[j] == Py_None) {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, j, Py_None);
      continue;
    }
    if (!THPVariable_Check(args[j])) {
      PyErr_Format(PyExc_TypeError, "expected a tensor or None, got %.100s", Py_TYPE(args[j])->tp_name);
      break;
    }
    const at::Tensor& t = THPVariable_Unpack(args[j]);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "this operator runs on CUDA tensors only");
      break;
    }
    if (t.layout() != at::kStrided || t.dim() < 1 || t.dim() > 4) {
      PyErr_SetString(PyExc_ValueError, "expected strided tensors of 1 to 4 dims");
      break;
    }
    const int on = t.get_device();
    if (device >= 0 && on != device) {
      PyErr_Format(PyExc_ValueError, "all tensors must be on cuda:%d (got one on cuda:%d)", device, on);
      break;
    }
    device = on;
    mssm_tensor& d = block[j - 1];
    d = mssm_tensor{};
    d.data = t.numel() > 0 ? t.data_ptr() : nullptr;
    d.dtype = dtype_of(t);
    d.ndim = int32_t(t.dim());
    for (int k = 0; k < int(t.dim()); ++k) {
      d.shape[k] = t.size(k);
      d.stride[k] = t.stride(k);
    }
    PyObject* at = PyLong_FromVoidPtr(&d);
    if (!at) break;
    PyTuple_SET_ITEM(out, j, at);
  }
  if (!PyErr_Occurred() && device < 0) PyErr_SetString(PyExc_ValueError, "no tensor given");
  PyObject* index = PyErr_Occurred() ? nullptr : PyLong_FromLong(device);
  if (!index) {
    Py_DECREF(out);
    return nullptr;
  }
  PyTuple_SET_ITEM(out, 0, index);
  return out;
}

// C++ exceptions (a tensor without storage) become Python ones
PyObject* describe_noexcept(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return describe(self, args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error while reading a tensor");
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"describe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(describe_noexcept)), METH_FASTCALL,
     "describe(block, *tensors) -> (device index, *addresses of the tensors' descriptors)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
