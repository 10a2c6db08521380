// The calls of packed.py from Python: argument checks, output allocation and
// the call of the C entry point, as in paged_binding.cpp, whose module they
// belong to.
#pragma once

#include <cmath>

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

// The sequences' borders.
const int* borders(PyObject* o, int device, int64_t* B) {
  const at::Tensor& cu = tensor(o, "cu");
  check_kind(cu, "cu", at::kInt, device);
  if (cu.dim() != 1 || cu.size(0) < 1 || !cu.is_contiguous())
    refuse(PyExc_ValueError, "cu has shape " + shape_of(cu) + ", expected contiguous [B + 1]");
  *B = cu.size(0) - 1;
  return static_cast<const int*>(cu.data_ptr());
}

// A row statistic [T, Hq].
float* statistic(const at::Tensor& t, const char* name, int64_t T, int64_t Hq, int device) {
  check_kind(t, name, at::kFloat, device);
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != Hq || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous [" + std::to_string(T) + ", " + std::to_string(Hq) + "]");
  return static_cast<float*>(t.data_ptr());
}

// The caller's workspace, or a new one of `need` bytes; its address (null where there is none) and size.
void* scratch(PyObject* given, size_t need, int device, at::Tensor* made, size_t* bytes) {
  if (given == Py_None) {
    *bytes = need;
    if (need == 0) return nullptr;
    *made = make({static_cast<int64_t>(need)}, at::kByte, device);
  } else {
    *made = tensor(given, "workspace");
    if (!made->is_cuda() || made->get_device() != device || !made->is_contiguous())
      refuse(PyExc_ValueError, "workspace must be contiguous on cuda:" + std::to_string(device));
    *bytes = made->nbytes();
  }
  return *bytes > 0 ? made->data_ptr() : nullptr;
}

// q, k and v of a call.
struct Packed {
  int device;
  const void *q, *k, *v;
  int64_t qs, ks, vs, T, Hq, Hkv, d, B;
  const int* cu;
  int t, hq, hkv, dd, b;
};

Packed packed_args(PyObject* qo, PyObject* ko, PyObject* vo, PyObject* cuo) {
  Packed p;
  p.device = device_of(qo, "q");
  const at::Tensor &q = tensor(qo, "q"), &k = tensor(ko, "k"), &v = tensor(vo, "v");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q has shape " + shape_of(q) + ", expected [T, heads, d]");
  p.T = q.size(0);
  p.Hq = q.size(1);
  p.d = q.size(2);
  p.qs = check_rows(q, "q", p.T, p.Hq, p.d, p.device);
  p.ks = check_rows(k, "k", p.T, -1, p.d, p.device);
  p.Hkv = k.size(1);
  p.vs = check_rows(v, "v", p.T, p.Hkv, p.d, p.device);
  p.cu = borders(cuo, p.device, &p.B);
  p.q = q.data_ptr();
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.t = small(p.T, "rows");
  p.hq = small(p.Hq, "heads");
  p.hkv = small(p.Hkv, "heads");
  p.dd = small(p.d, "d");
  p.b = small(p.B, "sequences");
  return p;
}

// The scale given, or 1 / sqrt(d).
double scale_of(PyObject* o, int64_t d) { return o == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(o); }

// packed_fwd(q, k, v, cu, causal, window, scale, out, lse, workspace) -> (out, lse)
PyObject* packed_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) refuse(PyExc_TypeError, "packed_fwd takes 10 arguments");
  const Packed p = packed_args(args[0], args[1], args[2], args[3]);
  const int causal = PyObject_IsTrue(args[4]);
  const long long window = PyLong_AsLongLong(args[5]);
  const double scale = scale_of(args[6], p.d);
  if (PyErr_Occurred()) return nullptr;
  int64_t os;
  at::Tensor o = rows_out(args[7], "out", p.T, p.Hq, p.d, p.device, &os), l, ws;
  if (!o.is_contiguous()) refuse(PyExc_ValueError, "out must be contiguous");
  l = args[8] == Py_None ? make({p.T, p.Hq}, at::kFloat, p.device) : tensor(args[8], "lse");
  float* lp = statistic(l, "lse", p.T, p.Hq, p.device);
  size_t bytes;
  void* wp = scratch(args[9], args[9] == Py_None ? fa_packed_fwd_workspace_bytes(p.b, p.t, p.hq, p.hkv, p.dd) : 0,
                     p.device, &ws, &bytes);
  void* op = o.data_ptr();
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.device)).stream();
  const int w = small(window, "window");
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = fa_packed_fwd(p.q, p.qs, p.k, p.ks, p.v, p.vs, p.cu, p.b, p.t, p.hq, p.hkv, p.dd, causal, w,
                       static_cast<float>(scale), op, lp, wp, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (failed(code, "fa_packed_fwd")) return nullptr;
  return tuple_of(output(args[7], o), output(args[8], l));
  END_HANDLE_TH_ERRORS
}

// packed_bwd(q, k, v, o, lse, do, cu, causal, window, scale, dq, dk, dv, workspace) -> (dq, dk, dv)
PyObject* packed_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) refuse(PyExc_TypeError, "packed_bwd takes 14 arguments");
  const Packed p = packed_args(args[0], args[1], args[2], args[6]);
  const at::Tensor &o = tensor(args[3], "o"), &l = tensor(args[4], "lse"), &g = tensor(args[5], "do");
  check_rows(o, "o", p.T, p.Hq, p.d, p.device);
  if (!o.is_contiguous()) refuse(PyExc_ValueError, "o must be contiguous");
  const float* lp = statistic(l, "lse", p.T, p.Hq, p.device);
  const int64_t gs = check_rows(g, "do", p.T, p.Hq, p.d, p.device);
  const int causal = PyObject_IsTrue(args[7]);
  const long long window = PyLong_AsLongLong(args[8]);
  const double scale = scale_of(args[9], p.d);
  if (PyErr_Occurred()) return nullptr;
  int64_t dqs, dks, dvs;
  at::Tensor dq = rows_out(args[10], "dq", p.T, p.Hq, p.d, p.device, &dqs),
             dk = rows_out(args[11], "dk", p.T, p.Hkv, p.d, p.device, &dks),
             dv = rows_out(args[12], "dv", p.T, p.Hkv, p.d, p.device, &dvs), ws;
  size_t bytes;
  void* wp = scratch(args[13], args[13] == Py_None ? fa_packed_bwd_workspace_bytes(p.b, p.t, p.hq, p.hkv, p.dd) : 0,
                     p.device, &ws, &bytes);
  const void *op = o.data_ptr(), *gp = g.data_ptr();
  void *dqp = dq.data_ptr(), *dkp = dk.data_ptr(), *dvp = dv.data_ptr();
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.device)).stream();
  const int w = small(window, "window");
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = fa_packed_bwd(p.q, p.qs, p.k, p.ks, p.v, p.vs, op, lp, gp, gs, p.cu, p.b, p.t, p.hq, p.hkv, p.dd, causal, w,
                       static_cast<float>(scale), dqp, dqs, dkp, dks, dvp, dvs, wp, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (failed(code, "fa_packed_bwd")) return nullptr;
  return tuple_of(output(args[10], dq), output(args[11], dk), output(args[12], dv));
  END_HANDLE_TH_ERRORS
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
