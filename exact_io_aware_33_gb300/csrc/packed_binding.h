// The calls of packed.py from Python: argument checks, output allocation and
// the call of the C entry point, as in paged_binding.cpp, whose module they
// belong to.
#pragma once

#include "binding_common.h"

namespace {

// The tensor an output goes to: the caller's, or a new one [rows, heads, d]; its row stride.
at::Tensor rows_out(PyObject* given, const char* name, int64_t rows, int64_t heads, int64_t d, int device,
                    int64_t* stride) {
  if (given == Py_None) {
    *stride = heads * d;
    return make({rows, heads, d}, at::kBFloat16, device);
  }
  const at::Tensor& t = tensor(given, name);
  *stride = check_rows(t, name, rows, heads, d, device);
  return t;
}

PyObject* output(PyObject* given, const at::Tensor& made) {
  return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given);
}

// Takes the references.
PyObject* tuple_of(PyObject* a, PyObject* b, PyObject* c = nullptr) {
  PyObject* all = !a || !b ? nullptr : c ? PyTuple_Pack(3, a, b, c) : PyTuple_Pack(2, a, b);
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return all;
}

int device_of(PyObject* q, const char* name) {
  const at::Tensor& t = tensor(q, name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (no CPU path exists)");
  return t.get_device();
}

// rope(q, k or None, positions, cos, sin, axis_of (bytes), interleaved, inverse, q_out, k_out) -> (q_out, k_out or None)
PyObject* rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) refuse(PyExc_TypeError, "rope takes 10 arguments");
  const int device = device_of(args[0], "q");
  const at::Tensor& q = tensor(args[0], "q");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q has shape " + shape_of(q) + ", expected [T, heads, d]");
  const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
  const int64_t qs = check_rows(q, "q", T, Hq, d, device);
  const at::Tensor &pos = tensor(args[2], "positions"), &c = tensor(args[3], "cos"), &s = tensor(args[4], "sin");
  check_kind(pos, "positions", at::kInt, device);
  if (pos.dim() != 2 || pos.size(1) != T || !pos.is_contiguous())
    refuse(PyExc_ValueError, "positions has shape " + shape_of(pos) + ", expected contiguous [axes, " + std::to_string(T) + "]");
  check_kind(c, "cos", at::kFloat, device);
  check_kind(s, "sin", at::kFloat, device);
  if (c.dim() != 2 || !c.sizes().equals(s.sizes()) || !c.is_contiguous() || !s.is_contiguous())
    refuse(PyExc_ValueError, "cos and sin must be contiguous [max_pos, rot / 2], both alike");
  if (!PyBytes_Check(args[5]) || PyBytes_GET_SIZE(args[5]) != c.size(1))
    refuse(PyExc_ValueError, "an axis is needed for each of the " + std::to_string(c.size(1)) + " pairs of cos and sin");
  const unsigned char* axes = reinterpret_cast<const unsigned char*>(PyBytes_AS_STRING(args[5]));
  const int interleaved = PyObject_IsTrue(args[6]), inverse = PyObject_IsTrue(args[7]);
  if (PyErr_Occurred()) return nullptr;
  int64_t qos = 0, ks = 0, kos = 0, Hk = 0;
  at::Tensor q_out = rows_out(args[8], "q_out", T, Hq, d, device, &qos), k_out;
  const void* kp = nullptr;
  void* kop = nullptr;
  if (args[1] != Py_None) {
    const at::Tensor& k = tensor(args[1], "k");
    ks = check_rows(k, "k", T, -1, d, device);
    Hk = k.size(1);
    k_out = rows_out(args[9], "k_out", T, Hk, d, device, &kos);
    kp = k.data_ptr();
    kop = k_out.data_ptr();
  } else if (args[9] != Py_None) {
    refuse(PyExc_ValueError, "k_out without k");
  }
  const void* qp = q.data_ptr();
  void* qop = q_out.data_ptr();
  const int* pp = static_cast<const int*>(pos.data_ptr());
  const float *cp = static_cast<const float*>(c.data_ptr()), *sp = static_cast<const float*>(s.data_ptr());
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  const int hq = small(Hq, "heads"), hk = small(Hk, "heads"), na = small(pos.size(0), "axes"), t = small(T, "rows"),
            mp = small(c.size(0), "max_pos"), rot = small(2 * c.size(1), "rot"), dd = small(d, "d");
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = fa_rope_axes(qp, qs, qop, qos, hq, kp, ks, kop, kos, hk, pp, na, t, axes, cp, sp, mp, rot, dd, interleaved,
                      inverse, stream);
  Py_END_ALLOW_THREADS;
  if (failed(code, "fa_rope_axes")) return nullptr;
  return tuple_of(output(args[8], q_out), args[1] == Py_None ? Py_NewRef(Py_None) : output(args[9], k_out));
  END_HANDLE_TH_ERRORS
}

}  // namespace
