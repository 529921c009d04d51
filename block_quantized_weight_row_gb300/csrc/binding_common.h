// binding_common.h — what the parts of the CPython extension share: exceptions
// for wrong arguments, tensors taken from them, the current stream.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdarg>

#include "bq.h"

namespace {

// What the caller got wrong, raised as a Python exception.
struct Wrong {
  PyObject *type;
};

[[noreturn]] void wrong(PyObject *type, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Wrong{type};
}

const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) wrong(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided) wrong(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}

int64_t to_int(PyObject *o, const char *name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) wrong(PyExc_TypeError, "%s must be an int", name);
  return v;
}

// A type, basis or other code that the library takes as an int.
int to_code(PyObject *o, const char *name) {
  const int64_t v = to_int(o, name);
  if (v < INT_MIN || v > INT_MAX) wrong(PyExc_ValueError, "%s must fit 32 bits", name);
  return int(v);
}

int elem_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return BQ_ELEM_F32;
    case at::kHalf: return BQ_ELEM_F16;
    case at::kBFloat16: return BQ_ELEM_BF16;
    default: return -1;
  }
}

void use_stream() { bq_set_stream(c10::cuda::getCurrentCUDAStream().stream()); }

PyObject *none() { Py_RETURN_NONE; }
PyObject *status(int r) { return PyLong_FromLong(r); }

// A workspace of this call's own, from the current stream's pool: calls on other
// streams and captured launches never share it. The one that the thread had set
// for other calls is set again at the end.
class CallWorkspace {
 public:
  CallWorkspace(size_t need, const at::Device &device)
      : ws_(at::empty({int64_t(std::max<size_t>(need, 256))}, at::TensorOptions().dtype(at::kByte).device(device))) {
    before_ = bq_get_workspace(&before_bytes_);
    bq_set_workspace(ws_.data_ptr(), size_t(ws_.numel()));
  }
  // (status, message) of the call just made, which stays the last message
  PyObject *failed(int r) {
    const std::string message = bq_last_error();
    restore();
    return Py_BuildValue("(is)", r, message.c_str());
  }
  ~CallWorkspace() { restore(); }

 private:
  void restore() {
    if (!restored_) bq_set_workspace(before_, before_bytes_);
    restored_ = true;
  }
  at::Tensor ws_;
  void *before_;
  size_t before_bytes_;
  bool restored_ = false;
};

}  // namespace
