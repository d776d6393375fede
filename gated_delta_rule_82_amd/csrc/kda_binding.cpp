// kda_binding.cpp - the call path of the Python binding (a CPython extension).
//
// A decode step of one user takes a few microseconds on the GPU; asking eleven
// tensors for pointer, dtype, shape, device and contiguity through Python takes
// ten.  This module reads them from the tensors themselves, fills the
// descriptors of include/kda.h and calls the entry point of libkda it is given.
// It holds no logic of its own: a tensor that cannot be passed makes call()
// return None, and the Python side says what is wrong.

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "kda.h"

namespace {

enum Kind { kRecurrence = 0, kPrefill = 1, kConv = 2, kWindow = 3, kVerify = 4 };
constexpr Py_ssize_t kTensors[] = {11, 11, 19, 17, 9};
constexpr int kMost = 19;

bool describe(PyObject* object, int64_t device, kda_tensor* d) {
  if (!THPVariable_Check(object)) return false;
  const at::Tensor& t = THPVariable_Unpack(object);
  if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device || !t.is_contiguous() || t.dim() > 4)
    return false;
  switch (t.scalar_type()) {
    case at::kFloat: d->dtype = KDA_F32; break;
    case at::kBFloat16: d->dtype = KDA_BF16; break;
    case at::kInt: d->dtype = KDA_I32; break;
    default: return false;
  }
  d->data = t.data_ptr();
  d->ndim = static_cast<int32_t>(t.dim());
  for (int i = 0; i < 4; ++i) d->shape[i] = i < d->ndim ? t.size(i) : 0;
  return true;
}

// call(kind, entry point, tensors, device, gate_mode, lower_bound, l2_eps,
//      scale, state_layout, matmul, stream) -> status, or None.
// tensors is a tuple in the entry point's order (None: draft_probs only).
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 11 || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "call: 11 arguments, the third a tuple");
    return nullptr;
  }
  const long kind = PyLong_AsLong(args[0]);
  void* const entry = PyLong_AsVoidPtr(args[1]);
  const long device = PyLong_AsLong(args[3]);
  kda_mode mode{};
  mode.gate_mode = static_cast<int32_t>(PyLong_AsLong(args[4]));
  mode.lower_bound = static_cast<float>(PyFloat_AsDouble(args[5]));
  mode.l2_eps = static_cast<float>(PyFloat_AsDouble(args[6]));
  mode.scale = static_cast<float>(PyFloat_AsDouble(args[7]));
  mode.state_layout = static_cast<int32_t>(PyLong_AsLong(args[8]));
  const long matmul = PyLong_AsLong(args[9]);
  hipStream_t const stream = static_cast<hipStream_t>(PyLong_AsVoidPtr(args[10]));
  if (PyErr_Occurred()) return nullptr;
  if (kind < 0 || kind > kVerify || PyTuple_GET_SIZE(args[2]) != kTensors[kind]) {
    PyErr_SetString(PyExc_TypeError, "call: wrong number of tensors");
    return nullptr;
  }
  kda_tensor t[kMost];
  const kda_tensor* p[kMost];
  try {
    for (Py_ssize_t i = 0; i < kTensors[kind]; ++i) {
      PyObject* const object = PyTuple_GET_ITEM(args[2], i);
      p[i] = t + i;
      if (kind == kVerify && i == 3 && object == Py_None) p[i] = nullptr;
      else if (!describe(object, device, t + i)) Py_RETURN_NONE;
    }
  } catch (...) {   // a tensor without storage of its own
    Py_RETURN_NONE;
  }
  int status = KDA_OK;
  Py_BEGIN_ALLOW_THREADS
  switch (kind) {
    case kRecurrence:
      status = reinterpret_cast<decltype(&kda_decode)>(entry)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8],
                                                              p[9], p[10], &mode, stream);
      break;
    case kPrefill:
      status = reinterpret_cast<decltype(&kda_prefill)>(entry)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8],
                                                               p[9], p[10], &mode, static_cast<int32_t>(matmul),
                                                               stream);
      break;
    case kConv: {
      const kda_conv conv = {t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], t[9], t[10], t[11]};
      status = reinterpret_cast<decltype(&kda_decode_conv)>(entry)(p[0], &conv, p[12], p[13], p[14], p[15], p[16],
                                                                   p[17], p[18], &mode, stream);
      break;
    }
    case kWindow: {
      const kda_replay replay = {t[11], t[12], t[13], t[14], t[15], t[16]};
      status = reinterpret_cast<decltype(&kda_decode_window)>(entry)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7],
                                                                     p[8], p[9], p[10], &replay, &mode, stream);
      break;
    }
    default:
      status = reinterpret_cast<decltype(&kda_verify)>(entry)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8],
                                                              stream);
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

PyMethodDef methods[] = {{"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
                          "call(kind, entry, tensors, device, gate_mode, lower_bound, l2_eps, scale, state_layout, "
                          "matmul, stream) -> status or None"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_binding", "The call path of the libkda binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_binding() { return PyModule_Create(&module); }
