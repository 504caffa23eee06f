// Shared by the extension's sources (attention_torch.cpp, adapters_torch.cpp): checks of
// tensors, the device and stream of a call, errors.  Not installed.
#pragma once

#include <ATen/MemoryOverlap.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "opq.h"

namespace opq_torch {

using at::Tensor;

extern PyObject* g_error;  // opq.OpqError

// The library launches on the current device: make it the tensors' one.
struct OnDevice {
  c10::DeviceIndex old, dev;
  explicit OnDevice(const Tensor& t) : old(c10::hip::current_device()), dev(t.device().index()) {
    if (old != dev) c10::hip::set_device(dev);
  }
  ~OnDevice() {
    if (old != dev) c10::hip::set_device(old);
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(dev).stream(); }
};

inline const Tensor& tensor_of(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name,
                    " must be a CUDA (HIP) tensor");
  return THPVariable_Unpack(o);
}

// These calls compute outside autograd: a result that ought to carry a gradient would
// come back without one, and nothing would say so.
inline const Tensor& plain(const Tensor& t, const char* name) {
  TORCH_CHECK(!(t.requires_grad() && at::GradMode::is_enabled()), name,
              " requires grad, which this call does not follow (apply_rotary, apply_linear and "
              "apply_adapted work under autograd): detach it, or call under torch.no_grad()");
  return t;
}
// A tensor whose memory this call writes: autograd learns of it, as of every in-place
// operation, should it have saved the old values.
inline void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A dense tensor of a known type and shape.
inline void* dense(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
            c10::Device dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.sizes() == shape && t.is_contiguous(), name,
                    " must be contiguous with shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be on ", dev, ", got ", t.device());
  return t.data_ptr();
}
inline void* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape,
            c10::Device dev) {
  return dense(tensor_of(o, name), name, type, shape, dev);
}

// A tensor whose last dimension is dense; its other strides are free.
inline const Tensor& rows(PyObject* o, const char* name, int64_t ndim) {
  const Tensor& t = tensor_of(o, name);
  TORCH_CHECK_VALUE(t.dim() == ndim && (t.size(-1) <= 1 || t.stride(-1) == 1), name, " must be ",
                    ndim, "-d with a dense last dimension");
  return plain(t, name);
}

inline int dtype_of(at::ScalarType t, const char* what) {
  TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, what,
                    " must be float32 or bfloat16, got ", t);
  return t == at::kFloat ? OPQ_F32 : OPQ_BF16;
}

inline void check(const char* fn, int status) {
  if (status == OPQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "sis", fn, status, opq_status_str(status));
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

inline int64_t int_of(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
inline double double_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

inline void arguments(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// A dense tensor of the allocator's on `like`'s device: what at::empty comes to, without the
// dispatcher and the options (pages_fork, with six of them: 7.8 to 6.7 us of host time).
inline Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), c10::nullopt);
}

// A workspace of the caller's, or of the allocator: of the current stream, so calls on
// different streams do not share one.
inline Tensor workspace_of(PyObject* o, size_t* bytes, const Tensor& like) {
  if (o == Py_None) {
    if (*bytes == 0) return Tensor();
    return fresh({(int64_t)*bytes}, at::kByte, like);
  }
  const Tensor& ws = tensor_of(o, "workspace");
  TORCH_CHECK_VALUE(ws.is_contiguous() && ws.device() == like.device(),
                    "workspace must be a contiguous tensor on ", like.device());
  *bytes = (size_t)ws.numel() * ws.element_size();
  return ws;
}

// adapters_torch.cpp
PyObject* lowrank_add(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* lowrank_backward(PyObject*, PyObject* const* a, Py_ssize_t n);

}  // namespace opq_torch
