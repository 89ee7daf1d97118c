// py_args.h -- what the Python bindings share: placing a call's arguments, and
// reading tensors.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

namespace py_args {
namespace {

using at::Tensor;

// Places positional and keyword arguments (a vectorcall's) in `out`, None as
// nullptr; the first `required` must be there.
template <int kCount>
bool place(const char* fn, const char* const (&names)[kCount], int required, PyObject* const* args, Py_ssize_t positional,
           PyObject* kwnames, PyObject* (&out)[kCount]) {
  for (PyObject*& o : out) o = nullptr;
  if (positional > kCount) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, kCount, positional);
    return false;
  }
  bool given[kCount] = {};
  for (Py_ssize_t i = 0; i < positional; ++i) {
    given[i] = true;
    out[i] = args[i] == Py_None ? nullptr : args[i];
  }
  const Py_ssize_t keywords = kwnames != nullptr ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t x = 0; x < keywords; ++x) {
    Py_ssize_t size = 0;
    const char* name = PyUnicode_AsUTF8AndSize(PyTuple_GET_ITEM(kwnames, x), &size);
    if (name == nullptr) return false;
    int i = 0;
    while (i < kCount && std::strcmp(names[i], name) != 0) ++i;
    if (i == kCount) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected keyword argument '%s'", fn, name);
      return false;
    }
    if (given[i]) {
      PyErr_Format(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, name);
      return false;
    }
    given[i] = true;
    PyObject* value = args[positional + x];
    out[i] = value == Py_None ? nullptr : value;
  }
  for (int i = 0; i < required; ++i)
    if (!given[i]) {
      PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
      return false;
    }
  return true;
}

const Tensor* tensor(PyObject* o, const char* what) {
  if (o != nullptr && THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
  return nullptr;
}

int64_t cuda_index(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

std::string shape_text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i > 0 ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

// Whether the tensor's storage holds it (it may have been made smaller, or been freed).
bool stored(const Tensor& t, const char* what) {
  if (t.numel() == 0) return true;
  int64_t extent = 1;
  for (int64_t i = 0; i < t.dim(); ++i) extent += (t.size(i) - 1) * t.stride(i);
  const uint64_t bytes = static_cast<uint64_t>(t.storage_offset() + extent) * t.element_size();
  if (t.storage().nbytes() >= bytes) return true;
  PyErr_Format(PyExc_ValueError, "the storage of %s is smaller than the tensor", what);
  return false;
}

template <class F>
PyCFunction as_function(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

}  // namespace
}  // namespace py_args
