// What the Python bindings share: checks of tensors, allocation of outputs, and
// how refusals and return codes become Python exceptions. Included by the one
// source file of the extension module.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstddef>
#include <string>

#include "fa.h"

namespace {

PyObject* g_fail = nullptr;  // paged.py's _check(code, what): raises FAError

// Raised as Python's TypeError or ValueError.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(PyObject* type, const std::string& text) { throw Refused{type, text}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void check_kind(const at::Tensor& t, const char* name, at::ScalarType dtype, int device) {
  if (t.is_cuda() && t.get_device() == device && t.scalar_type() == dtype) return;
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (no CPU path exists)");
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
  refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" +
                               std::to_string(device));
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t n : t.sizes()) s += std::to_string(n) + ", ";
  return s + ")";
}

// Checks a packed bf16 [rows, heads, d] tensor whose rows may lie apart (rows
// or heads below 0: any number of them); its row stride.
int64_t check_rows(const at::Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t d, int device) {
  check_kind(t, name, at::kBFloat16, device);
  if (t.dim() != 3 || t.size(2) != d || (rows >= 0 && t.size(0) != rows) || (heads >= 0 && t.size(1) != heads))
    refuse(PyExc_ValueError, std::string(name) + " has shape " + shape_of(t) + ", expected [" +
                                 (rows >= 0 ? std::to_string(rows) : "T") + ", " +
                                 (heads >= 0 ? std::to_string(heads) : "heads") + ", " + std::to_string(d) + "]");
  if (t.numel() == 0) return t.size(1) * d;
  if (t.stride(2) != 1 || (t.stride(1) != d && t.size(1) != 1))
    refuse(PyExc_ValueError, std::string("the heads and channels of ") + name + " must lie side by side");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * d;  // (one row: whatever its stride says)
}

at::Tensor make(at::IntArrayRef sizes, at::ScalarType dtype, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
}

template <typename T>
T* address(PyObject* o) {
  return static_cast<T*>(PyLong_AsVoidPtr(o));
}

int small(int64_t n, const char* what) {
  if (n < -0x7fffffff || n > 0x7fffffff) refuse(PyExc_ValueError, std::string(what) + " is out of range");
  return static_cast<int>(n);
}

bool failed(int code, const char* what) {
  if (code == FA_OK) return false;
  PyObject* r = PyObject_CallFunction(g_fail, "is", code, what);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: code %d", what, code);
  return true;
}

}  // namespace
