// The paged cache's calls from Python: argument checks, output allocation and
// the call of the C entry point, for paged.py.
//
// A step's small calls take 2 to 6 microseconds on the GPU, less than the
// interpreter and ctypes need for the same checks and allocations (10 to 12
// per call; here 5 to 6). Everything it does with tensors is read their
// metadata and allocate; the computation is the C library's.

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

// The batch for tensors of T rows.
fa_paged_batch batch_for(PyObject* o, int64_t T) {
  fa_paged_batch b = *address<const fa_paged_batch>(o);
  if (b.cu_q == nullptr && T != b.B)
    refuse(PyExc_ValueError, std::to_string(T) + " rows for " + std::to_string(b.B) + " sequences of one token each");
  if (T > 0x7fffffff) refuse(PyExc_ValueError, "too many rows");
  b.T = static_cast<int>(T);
  return b;
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

// The tensors that a struct's first fields were taken from, in that order.
constexpr const char* kCacheTensors[] = {"k_pages", "v_pages", "k_scales", "v_scales"};
constexpr const char* kBatchTensors[] = {"block_table", "kv_lens", "cu_q"};
static_assert(sizeof(void*) * 4 == offsetof(fa_paged_cache, num_pages) && sizeof(void*) * 3 == offsetof(fa_paged_batch, B));

// Refuses tensors that no longer lie where the struct says (their memory was
// replaced, and what the struct points at may be somebody else's).
template <typename S, size_t N>
void check_held(PyObject* held, const S* s, const char* const (&names)[N]) {
  const void* const* fields = reinterpret_cast<const void* const*>(s);
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = PyTuple_GET_ITEM(held, i);
    if (o != Py_None && tensor(o, names[i]).const_data_ptr() != fields[i])
      refuse(PyExc_ValueError, std::string("the memory of ") + names[i] + " has moved: make a new object for it");
  }
}

// attn(cache, its tensors, batch, its tensors, device, q, window, scale, out, lse, workspace) -> (out, lse)
PyObject* attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) refuse(PyExc_TypeError, "attn takes 11 arguments");
  const fa_paged_cache* cache = address<const fa_paged_cache>(args[0]);
  check_held(args[1], cache, kCacheTensors);
  check_held(args[3], address<const fa_paged_batch>(args[2]), kBatchTensors);
  const int device = static_cast<int>(PyLong_AsLong(args[4]));
  const at::Tensor& q = tensor(args[5], "q");
  const int64_t stride = check_rows(q, "q", -1, -1, cache->d, device), T = q.size(0), Hq = q.size(1);
  const fa_paged_batch batch = batch_for(args[2], T);
  const long long window = PyLong_AsLongLong(args[6]);
  const double scale = PyFloat_AsDouble(args[7]);
  if (PyErr_Occurred()) return nullptr;

  at::Tensor o, l, ws;
  if (args[8] == Py_None) {
    o = make({T, Hq, cache->d}, at::kBFloat16, device);
  } else {
    o = tensor(args[8], "out");
    check_rows(o, "out", T, Hq, cache->d, device);
    if (!o.is_contiguous()) refuse(PyExc_ValueError, "out must be contiguous");
  }
  if (args[9] == Py_None) {
    l = make({T, Hq}, at::kFloat, device);
  } else {
    l = tensor(args[9], "lse");
    check_kind(l, "lse", at::kFloat, device);
    if (l.dim() != 2 || l.size(0) != T || l.size(1) != Hq || !l.is_contiguous())
      refuse(PyExc_ValueError, "lse must be contiguous [" + std::to_string(T) + ", " + std::to_string(Hq) + "]");
  }
  size_t bytes = 0;
  if (args[10] == Py_None) {
    bytes = fa_paged_attn_workspace_bytes(cache, &batch, small(Hq, "heads"));
    if (bytes > 0) ws = make({static_cast<int64_t>(bytes)}, at::kByte, device);
  } else {
    ws = tensor(args[10], "workspace");
    if (!ws.is_cuda() || ws.get_device() != device || !ws.is_contiguous())
      refuse(PyExc_ValueError, "workspace must be contiguous on cuda:" + std::to_string(device));
    bytes = ws.nbytes();
  }
  const void* qp = q.data_ptr();
  void* op = o.data_ptr();
  float* lp = static_cast<float*>(l.data_ptr());
  void* wp = bytes > 0 ? ws.data_ptr() : nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  const int heads = small(Hq, "heads"), w = small(window, "window");
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = fa_paged_attn(cache, &batch, qp, stride, op, lp, heads, w, static_cast<float>(scale), wp, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (failed(code, "fa_paged_attn")) return nullptr;
  PyObject* a = args[8] == Py_None ? THPVariable_Wrap(o) : Py_NewRef(args[8]);
  PyObject* b = args[9] == Py_None ? THPVariable_Wrap(l) : Py_NewRef(args[9]);
  PyObject* both = PyTuple_Pack(2, a, b);
  Py_XDECREF(a);
  Py_XDECREF(b);
  return both;
  END_HANDLE_TH_ERRORS
}

// append(cache, its tensors, batch, its tensors, device, k, v, q, cos, sin, interleaved, q_out) -> q_out or None
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) refuse(PyExc_TypeError, "append takes 12 arguments");
  const fa_paged_cache* cache = address<const fa_paged_cache>(args[0]);
  check_held(args[1], cache, kCacheTensors);
  check_held(args[3], address<const fa_paged_batch>(args[2]), kBatchTensors);
  const int device = static_cast<int>(PyLong_AsLong(args[4]));
  const int64_t d = cache->d;
  const at::Tensor &k = tensor(args[5], "k"), &v = tensor(args[6], "v");
  const int64_t ks = check_rows(k, "k", -1, cache->num_heads, d, device), T = k.size(0);
  const int64_t vs = check_rows(v, "v", T, cache->num_heads, d, device);
  const fa_paged_batch batch = batch_for(args[2], T);
  const int interleaved = PyObject_IsTrue(args[10]);
  if (PyErr_Occurred()) return nullptr;

  const float *cos = nullptr, *sin = nullptr;
  int64_t max_pos = 0, rot = 0;
  if (args[8] != Py_None) {
    const at::Tensor &c = tensor(args[8], "cos"), &s = tensor(args[9], "sin");
    check_kind(c, "cos", at::kFloat, device);
    check_kind(s, "sin", at::kFloat, device);
    if (c.dim() != 2 || !c.sizes().equals(s.sizes()) || !c.is_contiguous() || !s.is_contiguous())
      refuse(PyExc_ValueError, "cos and sin must be contiguous [max_pos, rot / 2], both alike");
    max_pos = c.size(0);
    rot = 2 * c.size(1);
    cos = static_cast<const float*>(c.data_ptr());
    sin = static_cast<const float*>(s.data_ptr());
  }
  at::Tensor out;
  const void* qp = nullptr;
  void* op = nullptr;
  int64_t qs = 0, os = 0, Hq = 0;
  if (args[7] != Py_None) {
    const at::Tensor& q = tensor(args[7], "q");
    qs = check_rows(q, "q", T, -1, d, device);
    Hq = q.size(1);
    if (args[11] == Py_None) {
      out = make({T, Hq, d}, at::kBFloat16, device);
      os = Hq * d;
    } else {
      out = tensor(args[11], "q_out");
      os = check_rows(out, "q_out", T, Hq, d, device);
    }
    qp = q.data_ptr();
    op = out.data_ptr();
  }
  const void *kp = k.data_ptr(), *vp = v.data_ptr();
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  const int heads = small(Hq, "heads"), mp = small(max_pos, "max_pos"), r = small(rot, "rot");
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = fa_paged_append(cache, &batch, kp, ks, vp, vs, qp, qs, op, os, heads, cos, sin, mp, r, interleaved, stream);
  Py_END_ALLOW_THREADS;
  if (failed(code, "fa_paged_append")) return nullptr;
  if (args[7] == Py_None) Py_RETURN_NONE;
  return args[11] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(args[11]);
  END_HANDLE_TH_ERRORS
}

// END_HANDLE_TH_ERRORS turns C++ exceptions into Python's; a Refused carries its own type.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
}

PyObject* set_fail(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_fail, f);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {
    {"attn", fast(guarded<attn>), METH_FASTCALL, "fa_paged_attn on checked tensors"},
    {"append", fast(guarded<append>), METH_FASTCALL, "fa_paged_append on checked tensors"},
    {"set_fail", set_fail, METH_O, "the callable that raises a return code"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native() { return PyModule_Create(&g_module); }
