// The Python binding's fast part: writes a call's tensor descriptors, allocates its outputs and makes the call.
// A decode step is a few microseconds on the GPU; reading eight tensors' pointers, shapes and strides from
// Python takes longer than that.
#include <Python.h>

#include <algorithm>
#include <utility>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

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

// Fills `d` for a tensor and sets `device` or compares with it.  False: a Python error is set.
bool fill(PyObject* arg, mssm_tensor& d, int& device) {
  if (!THPVariable_Check(arg)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor, got %.100s", Py_TYPE(arg)->tp_name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(arg);
  if (!t.is_cuda()) {
    PyErr_SetString(PyExc_ValueError, "this operator runs on CUDA tensors only");
    return false;
  }
  if (t.layout() != at::kStrided || t.dim() < 1 || t.dim() > 4) {
    PyErr_SetString(PyExc_ValueError, "expected strided tensors of 1 to 4 dims");
    return false;
  }
  const int on = t.get_device();
  if (device >= 0 && on != device) {
    PyErr_Format(PyExc_ValueError, "all tensors must be on cuda:%d (got one on cuda:%d)", device, on);
    return false;
  }
  device = on;
  d = mssm_tensor{};
  d.data = t.numel() > 0 ? t.data_ptr() : nullptr;
  d.dtype = dtype_of(t);
  d.ndim = int32_t(t.dim());
  for (int k = 0; k < int(t.dim()); ++k) {
    d.shape[k] = t.size(k);
    d.stride[k] = t.stride(k);
  }
  return true;
}

// describe(block, *tensors) -> (device index, addresses): the descriptor of tensor j goes to block[j], and None
// stays None.  All tensors have to be on one CUDA device.
PyObject* describe(PyObject* const* args, Py_ssize_t n) {
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
  THPObjectPtr out(PyTuple_New(n));
  if (!out) return nullptr;
  for (Py_ssize_t j = 1; j < n; ++j) {
    PyObject* item = nullptr;
    if (args[j] == Py_None) {
      Py_INCREF(Py_None);
      item = Py_None;
    } else if (fill(args[j], block[j - 1], device)) {
      item = PyLong_FromVoidPtr(&block[j - 1]);
    }
    if (!item) return nullptr;
    PyTuple_SET_ITEM(out.get(), j, item);
  }
  PyObject* index = nullptr;
  if (device < 0) PyErr_SetString(PyExc_ValueError, "no tensor given");
  else index = PyLong_FromLong(device);
  if (!index) return nullptr;
  PyTuple_SET_ITEM(out.get(), 0, index);
  return out.release();
}

// Descriptors of a call's tensors, and the call itself, on a stream of their device.
struct Call {
  mssm_tensor d[20];
  int device = -1;
  int used = 0;
  c10::cuda::OptionalCUDAStreamGuard stream;
  // null for None; `ok` turns false with a Python error
  bool ok = true;
  const mssm_tensor* in(PyObject* arg) {
    if (!ok || arg == Py_None) return nullptr;
    ok = fill(arg, d[used], device);
    return ok ? &d[used++] : nullptr;
  }
  // A torch stream, a stream's address, or None for the device's current one: the outputs allocated from here on
  // belong to it.
  void on(PyObject* arg) {
    if (!ok || arg == Py_None || device < 0) return;
    THPObjectPtr address(PyIndex_Check(arg) ? PyNumber_Index(arg) : PyObject_GetAttrString(arg, "cuda_stream"));
    void* at = address ? PyLong_AsVoidPtr(address.get()) : nullptr;
    if (PyErr_Occurred()) ok = false;
    else stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(at), static_cast<c10::DeviceIndex>(device)));
  }
  // the output given, or a new one
  template <typename F>
  mssm_tensor* out(PyObject* arg, THPObjectPtr& made, F make) {
    if (!ok) return nullptr;
    if (arg == Py_None) {
      made = THPVariable_Wrap(make());
      if (!made) ok = false;
    } else {
      Py_INCREF(arg);
      made = arg;
    }
    return const_cast<mssm_tensor*>(ok ? in(made.get()) : nullptr);
  }
  // Owns `made`, as every reference here is owned: an allocation that fails part way raises a C++ exception, and
  // the outputs made before it must not outlive the call.
  template <typename F>
  PyObject* run(THPObjectPtr made, F f) {
    if (!ok) return nullptr;
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    void* at = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    mssm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f(at);
    Py_END_ALLOW_THREADS
    return st == MSSM_OK ? made.release() : PyLong_FromLong(long(st));
  }
};

// step(function, state, x, r, i, lam, r_bias, i_bias, z, decay scale, out, stream) -> out, or the status of a failed call
PyObject* step(PyObject* const* args, Py_ssize_t n) {
  if (n != 12) {
    PyErr_SetString(PyExc_TypeError, "step takes 12 arguments");
    return nullptr;
  }
  const auto fn = reinterpret_cast<decltype(&mssm_gated_state_update)>(PyLong_AsVoidPtr(args[0]));
  const double c = PyFloat_AsDouble(args[9]);
  if (!fn || PyErr_Occurred()) return nullptr;
  Call call;
  auto* state = const_cast<mssm_tensor*>(call.in(args[1]));
  const mssm_tensor *x = call.in(args[2]), *r = call.in(args[3]), *i = call.in(args[4]), *lam = call.in(args[5]),
                    *rb = call.in(args[6]), *ib = call.in(args[7]), *z = call.in(args[8]);
  THPObjectPtr made;
  if (call.ok && !x) {
    PyErr_SetString(PyExc_TypeError, "x: expected a tensor");
    return nullptr;
  }
  call.on(args[11]);
  mssm_tensor* out = call.out(args[10], made, [&] {
    const at::Tensor& t = THPVariable_Unpack(args[2]);
    return at::empty(t.sizes(), t.options().requires_grad(false));
  });
  return call.run(std::move(made), [&](void* s) { return fn(state, x, r, i, lam, rb, ib, z, float(c), out, s); });
}

// scan(function, x, r, i, lam, r_bias, i_bias, z, decay scale, h0, cu_seqlens, out, last_state, whether to return it,
// stream) -> (out, last_state), or the status of a failed call
PyObject* scan(PyObject* const* args, Py_ssize_t n) {
  if (n != 15) {
    PyErr_SetString(PyExc_TypeError, "scan takes 15 arguments");
    return nullptr;
  }
  const auto fn = reinterpret_cast<decltype(&mssm_gated_scan_fwd)>(PyLong_AsVoidPtr(args[0]));
  const double c = PyFloat_AsDouble(args[8]);
  const int want = PyObject_IsTrue(args[13]);
  if (!fn || want < 0 || PyErr_Occurred()) return nullptr;
  Call call;
  const mssm_tensor* t[7];
  for (int k = 0; k < 7; ++k) t[k] = call.in(args[1 + k]);
  const mssm_gated_ext ext{int32_t(sizeof(mssm_gated_ext)), float(c), call.in(args[9]), call.in(args[10])};
  if (!call.ok) return nullptr;
  if (!t[0] || t[0]->ndim != 3) {
    PyErr_SetString(PyExc_ValueError, "x: expected [Bt, D, L]");
    return nullptr;
  }
  const at::Tensor& x = THPVariable_Unpack(args[1]);
  const int64_t seqs = ext.cu_seqlens ? std::max<int64_t>(ext.cu_seqlens->shape[0] - 1, 0) : x.size(0);
  call.on(args[14]);
  if (!call.ok) return nullptr;
  THPObjectPtr both(PyTuple_New(2)), out_made, last_made;
  if (!both) return nullptr;
  mssm_tensor* out = call.out(args[11], out_made, [&] { return at::empty(x.sizes(), x.options().requires_grad(false)); });
  PyTuple_SET_ITEM(both.get(), 0, out_made.release());
  mssm_tensor* last = nullptr;
  if (want || args[12] != Py_None) {
    last = call.out(args[12], last_made, [&] {
      return at::empty({seqs, x.size(1)}, x.options().dtype(at::kFloat).requires_grad(false));
    });
  } else {
    Py_INCREF(Py_None);
    last_made = Py_None;
  }
  PyTuple_SET_ITEM(both.get(), 1, last_made.release());
  return call.run(std::move(both), [&](void* s) { return fn(t[0], t[1], t[2], t[3], t[4], t[5], t[6], &ext, out, last, s); });
}

// scan_bwd(function, x, r, i, lam, r_bias, i_bias, z, decay scale, h0, cu_seqlens, dout, dlast_state, stream) ->
// (dx, dr, di, dz, dlam, dr_bias, di_bias, dh0), or the status of a failed call
PyObject* scan_bwd(PyObject* const* args, Py_ssize_t n) {
  if (n != 14) {
    PyErr_SetString(PyExc_TypeError, "scan_bwd takes 14 arguments");
    return nullptr;
  }
  const auto fn = reinterpret_cast<decltype(&mssm_gated_scan_bwd)>(PyLong_AsVoidPtr(args[0]));
  const double c = PyFloat_AsDouble(args[8]);
  if (!fn || PyErr_Occurred()) return nullptr;
  Call call;
  const mssm_tensor* t[7];
  for (int k = 0; k < 7; ++k) t[k] = call.in(args[1 + k]);
  const mssm_gated_ext ext{int32_t(sizeof(mssm_gated_ext)), float(c), call.in(args[9]), call.in(args[10])};
  const mssm_tensor *dout = call.in(args[11]), *dlast = call.in(args[12]);
  if (!call.ok) return nullptr;
  if (!t[0] || t[0]->ndim != 3) {
    PyErr_SetString(PyExc_ValueError, "x: expected [Bt, D, L]");
    return nullptr;
  }
  const at::Tensor& x = THPVariable_Unpack(args[1]);
  const auto like = x.options().requires_grad(false), f32 = like.dtype(at::kFloat);
  call.on(args[13]);
  if (!call.ok) return nullptr;
  THPObjectPtr made(PyTuple_New(8));
  if (!made) return nullptr;
  mssm_tensor* g[8];
  for (int k = 0; k < 8; ++k) {
    // dz, the biases' gradients and dh0 come with their inputs
    const bool on = k == 3 ? t[6] != nullptr : k == 5 ? t[4] != nullptr : k == 6 ? t[5] != nullptr : k == 7 ? ext.h0 != nullptr : true;
    THPObjectPtr one;
    if (on) {
      g[k] = call.out(Py_None, one, [&] {
        if (k < 4) return at::empty(x.sizes(), like);
        if (k < 7) return at::empty({x.size(1)}, f32);
        return at::empty(THPVariable_Unpack(args[9]).sizes(), f32);
      });
    } else {
      g[k] = nullptr;
      Py_INCREF(Py_None);
      one = Py_None;
    }
    PyTuple_SET_ITEM(made.get(), k, one.release());
  }
  mssm_tensor ws{};
  at::Tensor sums;
  if (x.size(0) > 1) {
    sums = at::empty({3, x.size(0), x.size(1)}, f32);
    ws = mssm_tensor{sums.numel() ? sums.data_ptr() : nullptr, MSSM_F32, 3, {3, x.size(0), x.size(1), 0},
                     {sums.stride(0), sums.stride(1), sums.stride(2), 0}};
  }
  return call.run(std::move(made), [&](void* s) {
    return fn(t[0], t[1], t[2], t[3], t[4], t[5], t[6], &ext, dout, dlast, g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7],
              sums.defined() ? &ws : nullptr, s);
  });
}

// linear(function, x, qweight, qscales, qzeros, group, bias, outputs, out, stream) -> out, or the status of a failed call
PyObject* linear(PyObject* const* args, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "linear takes 10 arguments");
    return nullptr;
  }
  const auto fn = reinterpret_cast<decltype(&mssm_w4_linear)>(PyLong_AsVoidPtr(args[0]));
  const int64_t group = PyLong_AsLongLong(args[5]), outputs = PyLong_AsLongLong(args[7]);
  if (!fn || PyErr_Occurred()) return nullptr;
  Call call;
  const mssm_tensor *x = call.in(args[1]), *q = call.in(args[2]), *s = call.in(args[3]), *z = call.in(args[4]),
                    *b = call.in(args[6]);
  THPObjectPtr made;
  if (call.ok && !x) {
    PyErr_SetString(PyExc_TypeError, "x: expected a tensor");
    return nullptr;
  }
  call.on(args[9]);
  mssm_tensor* out = call.out(args[8], made, [&] {
    const at::Tensor& t = THPVariable_Unpack(args[1]);
    return at::empty({t.size(0), outputs}, t.options().requires_grad(false));
  });
  return call.run(std::move(made), [&](void* stream) { return fn(x, q, s, z, group, b, out, stream); });
}

// C++ exceptions (out of memory, a tensor without storage) become the Python ones that torch raises
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(args, n);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<F>));
}

PyMethodDef methods[] = {
    {"describe", method<describe>(), METH_FASTCALL, "describe(block, *tensors) -> (device index, *descriptor addresses)"},
    {"step", method<step>(), METH_FASTCALL,
     "step(function, state, x, r, i, lam, r_bias, i_bias, z, decay_scale, out, stream) -> out, or a failed call's status"},
    {"scan", method<scan>(), METH_FASTCALL,
     "scan(function, x, r, i, lam, r_bias, i_bias, z, decay_scale, h0, cu_seqlens, out, last_state, want_last, stream) -> "
     "(out, last_state), or a failed call's status"},
    {"scan_bwd", method<scan_bwd>(), METH_FASTCALL,
     "scan_bwd(function, x, r, i, lam, r_bias, i_bias, z, decay_scale, h0, cu_seqlens, dout, dlast_state, stream) -> gradients, or "
     "a failed call's status"},
    {"linear", method<linear>(), METH_FASTCALL,
     "linear(function, x, qweight, qscales, qzeros, group, bias, outputs, out, stream) -> out, or a failed call's status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
