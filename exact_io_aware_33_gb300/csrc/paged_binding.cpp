// The paged cache's calls from Python: argument checks, output allocation and
// the call of the C entry point, for paged.py; and the extension module, which
// also holds the calls of packed_binding.h, for packed.py.
//
// A step's small calls take 2 to 6 microseconds on the GPU, less than the
// interpreter and ctypes need for the same checks and allocations (10 to 12
// per call; here 5 to 6). Everything it does with tensors is read their
// metadata and allocate; the computation is the C library's.

#include "binding_common.h"
#include "packed_binding.h"

namespace {

// The batch for tensors of T rows.
fa_paged_batch batch_for(PyObject* o, int64_t T) {
  fa_paged_batch b = *address<const fa_paged_batch>(o);
  if (b.cu_q == nullptr && T != b.B)
    refuse(PyExc_ValueError, std::to_string(T) + " rows for " + std::to_string(b.B) + " sequences of one token each");
  if (T > 0x7fffffff) refuse(PyExc_ValueError, "too many rows");
  b.T = static_cast<int>(T);
  return b;
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
    {"packed_fwd", fast(guarded<packed_fwd>), METH_FASTCALL, "fa_packed_fwd on checked tensors"},
    {"packed_bwd", fast(guarded<packed_bwd>), METH_FASTCALL, "fa_packed_bwd on checked tensors"},
    {"rope", fast(guarded<rope>), METH_FASTCALL, "fa_rope_axes on checked tensors"},
    {"set_fail", set_fail, METH_O, "the callable that raises a return code"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native() { return PyModule_Create(&g_module); }
