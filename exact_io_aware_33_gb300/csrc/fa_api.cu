// C ABI of libfa.so: argument checks, TMA tensor maps, the device status
// word, and the extern "C" entry points declared in fa.h.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// One status word per device: set by a kernel whose bounded wait ran out.
__device__ int g_status_word;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kSmemSlots = 48;

struct DeviceState {
  bool probed = false;
  bool supported = false;
  int sms = 0;
  int* status = nullptr;
  bool smem_set[kSmemSlots] = {};
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

EncodeTiledFn encode_fn() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  return g_encode;
}

// Current device, checked once: compute capability 10.3 (GB300).
int current_device(DeviceState** st) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState& s = g_dev[dev];
  if (!s.probed) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return FA_ERR_LAUNCH;
    s.supported = (major == 10 && minor == 3);
    if (cudaDeviceGetAttribute(&s.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FA_ERR_LAUNCH;
    void* addr = nullptr;
    if (s.supported) {
      if (cudaGetSymbolAddress(&addr, g_status_word) != cudaSuccess) return FA_ERR_LAUNCH;
      s.status = static_cast<int*>(addr);
    }
    s.probed = true;
  }
  *st = &s;
  return s.supported ? FA_OK : FA_ERR_UNSUPPORTED;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// Common checks of both passes. Returns FA_OK, or an error code; sets
// *empty when there is nothing to compute.
int check_problem(int B, int H, int N, int d, float scale, bool* empty) {
  *empty = false;
  if (B < 0 || H < 0 || N < 0) return FA_ERR_INVALID;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || N == 0) {
    *empty = true;
    return FA_OK;
  }
  const long long bh = static_cast<long long>(B) * H;
  if (bh > (1LL << 31) - 1) return FA_ERR_INVALID;
  // TMA coordinates and tensor extents are 32-bit; keep element offsets in range.
  if (bh * static_cast<long long>(N) * d > (1LL << 46)) return FA_ERR_INVALID;
  return FA_OK;
}

bool make_map_bhnd(CUtensorMap* map, const void* ptr, int BH, int N, int d, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool make_map_pages(CUtensorMap* map, const void* ptr, int blocks, int rows, int d, int box_rows, bool swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d),
                                 static_cast<cuuint64_t>(rows) * static_cast<cuuint64_t>(d)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE,
          !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool make_map_packed(CUtensorMap* map, const void* ptr, int T, int heads, int group, int d, long long row_stride,
                     int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(group),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(group) * static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(group), 1, static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int current_device_status() {
  DeviceState* st = nullptr;
  return current_device(&st);
}

int* device_status_word() {
  DeviceState* st = nullptr;
  if (current_device(&st) != FA_OK) return nullptr;
  return st->status;
}

int device_sm_count() {
  DeviceState* st = nullptr;
  if (current_device(&st) != FA_OK) return 0;
  return st->sms;
}

bool ensure_smem_attr(const void* func, int bytes, int slot) {
  DeviceState* st = nullptr;
  if (current_device(&st) != FA_OK || slot < 0 || slot >= kSmemSlots) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!st->smem_set[slot]) {
    if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
      return false;
    st->smem_set[slot] = true;
  }
  return true;
}

}  // namespace fa

using fa::Problem;

extern "C" {

int fa_version(void) { return 100; }

const char* fa_strerror(int code) {
  switch (code) {
    case FA_OK: return "success";
    case FA_ERR_INVALID: return "invalid argument (pointer, size, alignment or scale)";
    case FA_ERR_UNSUPPORTED:
      return "unsupported (head size 64 or 128, or 256 in the forward; device must be CC 10.3)";
    case FA_ERR_LAUNCH: return "a CUDA call failed (launch, attribute or tensor map)";
    case FA_ERR_TIMEOUT: return "a bounded wait inside a kernel ran out";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_INDEX: return "a page, length, row range or position read on the device was out of range";
    default: return "unknown error code";
  }
}

int fa_fwd_stream(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                  int N, int d, int causal, float scale, void* cuda_stream) {
  bool empty = false;
  int rc = fa::check_problem(B, H, N, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!fa::aligned16(q) || !fa::aligned16(k) || !fa::aligned16(v) || !fa::aligned16(o) ||
      !fa::aligned16(lse))
    return FA_ERR_INVALID;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  Problem p{q, k, v, B, H, N, d, causal, scale};
  return fa::launch_fwd(p, o, lse, static_cast<cudaStream_t>(cuda_stream));
}

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
           int d, int causal, float scale) {
  return fa_fwd_stream(q, k, v, o, lse, B, H, N, d, causal, scale, nullptr);
}

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d) {
  if (B <= 0 || H <= 0 || N <= 0 || d <= 0) return 0;
  return fa::bwd_workspace_bytes(B, H, N, d);
}

namespace {

// Checks shared by the backward entry points. `ptrs` must all be non-NULL
// and 16-byte aligned; the workspace 256-byte aligned and large enough.
int check_bwd(int B, int H, int N, int d, float scale, std::initializer_list<const void*> ptrs,
              const void* workspace, size_t ws_bytes, bool* empty) {
  int rc = fa::check_problem(B, H, N, d, scale, empty);
  if (rc != FA_OK || *empty) return rc;
  if (d == 256) return FA_ERR_UNSUPPORTED;  // the backward's accumulators need d <= 128
  for (const void* ptr : ptrs)
    if (!fa::aligned16(ptr)) return FA_ERR_INVALID;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      ws_bytes < fa::bwd_workspace_bytes(B, H, N, d))
    return FA_ERR_WORKSPACE;
  fa::DeviceState* st = nullptr;
  return fa::current_device(&st);
}

}  // namespace

int fa_bwd_preprocess_stream(const void* o, const float* lse, const void* dO, int B, int H,
                             int N, int d, void* workspace, size_t ws_bytes, void* cuda_stream) {
  bool empty = false;
  int rc = check_bwd(B, H, N, d, 1.f, {o, lse, dO}, workspace, ws_bytes, &empty);
  if (rc != FA_OK || empty) return rc;
  Problem p{nullptr, nullptr, nullptr, B, H, N, d, 0, 1.f};
  return fa::launch_bwd_pre(p, o, lse, dO, workspace, static_cast<cudaStream_t>(cuda_stream));
}

int fa_bwd_main_stream(const void* q, const void* k, const void* v, const void* dO, void* dk,
                       void* dv, int B, int H, int N, int d, int causal, float scale,
                       void* workspace, size_t ws_bytes, void* cuda_stream) {
  bool empty = false;
  int rc = check_bwd(B, H, N, d, scale, {q, k, v, dO, dk, dv}, workspace, ws_bytes, &empty);
  if (rc != FA_OK || empty) return rc;
  Problem p{q, k, v, B, H, N, d, causal, scale};
  return fa::launch_bwd_main(p, dO, dk, dv, workspace, static_cast<cudaStream_t>(cuda_stream));
}

int fa_bwd_finish_stream(void* dq, int B, int H, int N, int d, const void* workspace,
                         size_t ws_bytes, void* cuda_stream) {
  bool empty = false;
  int rc = check_bwd(B, H, N, d, 1.f, {dq}, workspace, ws_bytes, &empty);
  if (rc != FA_OK || empty) return rc;
  Problem p{nullptr, nullptr, nullptr, B, H, N, d, 0, 1.f};
  return fa::launch_bwd_post(p, dq, workspace, static_cast<cudaStream_t>(cuda_stream));
}

int fa_bwd_stream(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                  int causal, float scale, void* workspace, size_t ws_bytes, void* cuda_stream) {
  bool empty = false;
  int rc = check_bwd(B, H, N, d, scale, {q, k, v, o, lse, dO, dq, dk, dv}, workspace, ws_bytes,
                     &empty);
  if (rc != FA_OK || empty) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  Problem p{q, k, v, B, H, N, d, causal, scale};
  rc = fa::launch_bwd_pre(p, o, lse, dO, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_main(p, dO, dk, dv, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_post(p, dq, workspace, st);
  return rc;
}

int fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const float* lse,
              const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
              int d_v, int causal, int window, float scale, void* workspace, size_t ws_bytes,
              void* cuda_stream) {
  if (window < 0 || (window > 0 && !causal)) return FA_ERR_INVALID;
  if (d_v != 64 && d_v != 128) return FA_ERR_UNSUPPORTED;
  bool empty = false;
  int rc = check_bwd(B, H, N, d, scale, {q, k, v, o, lse, dO, dq, dk, dv}, workspace, ws_bytes,
                     &empty);
  if (rc != FA_OK || empty) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  Problem p{q, k, v, B, H, N, d, causal, scale, window, d_v};
  rc = fa::launch_bwd_pre(p, o, lse, dO, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_main(p, dO, dk, dv, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_post(p, dq, workspace, st);
  return rc;
}

namespace {

// Dropout parameters after checks: FA_ERR_INVALID unless 0 <= p < 1.
int make_dropout(float p, unsigned long long seed, unsigned long long offset, fa::Dropout* out) {
  if (!(p >= 0.f && p < 1.f)) return FA_ERR_INVALID;
  long t = lrintf(256.f * p);
  if (t > 255) t = 255;
  out->t = static_cast<uint32_t>(t);
  out->inv_keep = 256.f / static_cast<float>(256 - t);
  out->seed_lo = static_cast<uint32_t>(seed & 0xffffffffull);
  out->seed_hi = static_cast<uint32_t>(seed >> 32);
  out->offset = static_cast<uint32_t>(offset & 0xffffffffull);
  return FA_OK;
}

}  // namespace

int fa_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                   int N, int d, int causal, float scale, float dropout_p, unsigned long long seed,
                   unsigned long long offset, void* cuda_stream) {
  fa::Dropout drop;
  int rc = make_dropout(dropout_p, seed, offset, &drop);
  if (rc != FA_OK) return rc;
  bool empty = false;
  rc = fa::check_problem(B, H, N, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!fa::aligned16(q) || !fa::aligned16(k) || !fa::aligned16(v) || !fa::aligned16(o) ||
      !fa::aligned16(lse))
    return FA_ERR_INVALID;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  Problem p{q, k, v, B, H, N, d, causal, scale};
  p.drop = drop;
  return fa::launch_fwd(p, o, lse, static_cast<cudaStream_t>(cuda_stream));
}

int fa_bwd_dropout(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   int causal, float scale, float dropout_p, unsigned long long seed,
                   unsigned long long offset, void* workspace, size_t ws_bytes, void* cuda_stream) {
  fa::Dropout drop;
  int rc = make_dropout(dropout_p, seed, offset, &drop);
  if (rc != FA_OK) return rc;
  bool empty = false;
  rc = check_bwd(B, H, N, d, scale, {q, k, v, o, lse, dO, dq, dk, dv}, workspace, ws_bytes, &empty);
  if (rc != FA_OK || empty) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  Problem p{q, k, v, B, H, N, d, causal, scale};
  p.drop = drop;
  rc = fa::launch_bwd_pre(p, o, lse, dO, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_main(p, dO, dk, dv, workspace, st);
  if (rc == FA_OK) rc = fa::launch_bwd_post(p, dq, workspace, st);
  return rc;
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
           const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, int causal,
           float scale) {
  bool empty = false;
  int rc = fa::check_problem(B, H, N, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (d == 256) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!fa::aligned16(ptr)) return FA_ERR_INVALID;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  const size_t bytes = fa::bwd_workspace_bytes(B, H, N, d);
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, bytes, nullptr) != cudaSuccess) return FA_ERR_LAUNCH;
  rc = fa_bwd_stream(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, causal, scale, ws, bytes,
                     nullptr);
  if (cudaFreeAsync(ws, nullptr) != cudaSuccess && rc == FA_OK) rc = FA_ERR_LAUNCH;
  return rc;
}

namespace {

// Checks of the extended forward forms; sets *empty for B, H or Nq = 0.
int check_fwd_ex(int B, int H, int Nq, int Nk, int d, int dv, int causal, int window, float scale,
                 std::initializer_list<const void*> ptrs, bool* empty) {
  *empty = false;
  if (B < 0 || H < 0 || Nq < 0 || Nk < 0 || window < 0) return FA_ERR_INVALID;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID;
  // (d, dv) in {64, 128}^2, or d = dv = 256
  if (!(d == 256 && dv == 256) && ((d != 64 && d != 128) || (dv != 64 && dv != 128)))
    return FA_ERR_UNSUPPORTED;
  if (window > 0 && !causal) return FA_ERR_INVALID;
  if (B == 0 || H == 0 || Nq == 0) {
    *empty = true;
    return FA_OK;
  }
  if (Nk == 0 || (causal && Nq > Nk)) return FA_ERR_INVALID;
  const long long bh = static_cast<long long>(B) * H;
  if (bh > (1LL << 31) - 1) return FA_ERR_INVALID;
  if (bh * static_cast<long long>(Nq > Nk ? Nq : Nk) * (d > dv ? d : dv) > (1LL << 46))
    return FA_ERR_INVALID;
  for (const void* ptr : ptrs)
    if (!fa::aligned16(ptr)) return FA_ERR_INVALID;
  fa::DeviceState* st = nullptr;
  return fa::current_device(&st);
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 148;
}

}  // namespace

int fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int Nq, int Nk, int d, int dv, int causal, int window, float scale,
              void* cuda_stream) {
  bool empty = false;
  int rc = check_fwd_ex(B, H, Nq, Nk, d, dv, causal, window, scale, {q, k, v, o, lse}, &empty);
  if (rc != FA_OK || empty) return rc;
  fa::FwdProblem p{q, k, v, B, H, Nq, Nk, d, dv, causal, window, scale};
  return fa::launch_fwd_general(p, o, lse, nullptr, nullptr, 1,
                                static_cast<cudaStream_t>(cuda_stream));
}

int fa_decode_num_splits(int B, int H, int Nq, int Nk, int n_splits) {
  if (B <= 0 || H <= 0 || Nq <= 0 || Nk <= 0) return 0;
  fa::FwdProblem p{nullptr, nullptr, nullptr, B, H, Nq, Nk, 64, 64, 0, 0, 1.f};
  return fa::fwd_split_count(p, n_splits, sm_count());
}

size_t fa_decode_workspace_bytes(int B, int H, int Nq, int Nk, int dv, int n_splits) {
  const int s = fa_decode_num_splits(B, H, Nq, Nk, n_splits);
  if (s <= 0 || dv <= 0) return 0;
  return static_cast<size_t>(s) * B * H * Nq * (static_cast<size_t>(dv) + 1) * 4;
}

int fa_decode_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                      int H, int Nq, int Nk, int d, int dv, int causal, int window, float scale,
                      int n_splits, void* workspace, size_t ws_bytes, void* cuda_stream) {
  bool empty = false;
  int rc = check_fwd_ex(B, H, Nq, Nk, d, dv, causal, window, scale, {q, k, v, o, lse}, &empty);
  if (rc != FA_OK || empty) return rc;
  const size_t need = fa_decode_workspace_bytes(B, H, Nq, Nk, dv, n_splits);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < need)
    return FA_ERR_WORKSPACE;
  const int s = fa_decode_num_splits(B, H, Nq, Nk, n_splits);
  fa::FwdProblem p{q, k, v, B, H, Nq, Nk, d, dv, causal, window, scale};
  float* part_o = static_cast<float*>(workspace);
  float* part_lse = part_o + static_cast<size_t>(s) * B * H * Nq * dv;
  return fa::launch_fwd_general(p, o, lse, part_o, part_lse, s,
                                static_cast<cudaStream_t>(cuda_stream));
}

namespace {

bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks of the cache and the batch that both paged entry points share; fills
// the internal forms. *empty: no sequence or no row, nothing is read.
int check_paged(const fa_paged_cache* c, const fa_paged_batch* b, fa::PagedPool* pool,
                fa::PagedBatchDev* dev, bool* empty) {
  *empty = false;
  if (c == nullptr || b == nullptr) return FA_ERR_INVALID;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  const int ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128) return FA_ERR_UNSUPPORTED;
  if (c->num_pages < 0 || c->num_heads <= 0 || b->B < 0 || b->T < 0 || b->max_q < 1 || b->max_pages < 0 ||
      b->max_kv < 0)
    return FA_ERR_INVALID;
  if (b->B == 0 || b->T == 0) {
    *empty = true;
    return FA_OK;
  }
  if (b->cu_q == nullptr && (b->T != b->B || b->max_q != 1)) return FA_ERR_INVALID;
  if (c->num_pages == 0 || b->max_pages == 0) return FA_ERR_INVALID;
  // tensor-map coordinates and positions are 32-bit
  if (static_cast<long long>(c->num_pages) * c->num_heads > 0x7fffffffLL) return FA_ERR_INVALID;
  if (static_cast<long long>(b->max_pages) * ps > 0x7fffffffLL - 4096) return FA_ERR_INVALID;  // (and tiles ahead)
  if (!fa::aligned16(c->k_pages) || !fa::aligned16(c->v_pages) || !aligned4(c->k_scales) ||
      !aligned4(c->v_scales) || !aligned4(b->block_table) || !aligned4(b->kv_lens) ||
      (b->cu_q != nullptr && !aligned4(b->cu_q)))
    return FA_ERR_INVALID;
  *pool = fa::PagedPool{c->k_pages, c->v_pages, c->k_scales, c->v_scales,
                        c->num_pages, c->num_heads, ps, c->d};
  int shift = 4;
  while ((1 << shift) < ps) ++shift;
  *dev = fa::PagedBatchDev{b->block_table, b->kv_lens, b->cu_q, b->B, b->T, b->max_q, b->max_pages,
                           ps, shift, c->num_pages};
  return FA_OK;
}

// Rows of `heads` x d elements, `stride` elements apart, read in 16-byte words.
bool row_stride_ok(long long stride, int heads, int d) {
  return stride >= static_cast<long long>(heads) * d && stride % 8 == 0 && stride <= (1LL << 40);
}

// Whether two packed bf16 tensors of T rows share memory: rows of `aw` and `bw`
// elements, `as` and `bs` elements apart. Exact where the strides are equal
// (slices of one fused projection interleave without meeting).
bool rows_meet(const void* a, long long as, long long aw, const void* b, long long bs, long long bw, int T) {
  const long long a0 = static_cast<long long>(reinterpret_cast<uintptr_t>(a)), b0 = static_cast<long long>(reinterpret_cast<uintptr_t>(b));
  if (a0 + 2 * ((T - 1) * as + aw) <= b0 || b0 + 2 * ((T - 1) * bs + bw) <= a0) return false;
  if (T == 1 || as != bs) return true;
  const long long off = (b0 - a0) % (2 * as), ahead = off < 0 ? off + 2 * as : off;  // of a's nearest row before it
  return ahead < 2 * aw || ahead + 2 * bw > 2 * as;
}

// Whether T rows of aw 16-bit elements, as elements apart, share bytes with the `bytes` from b on.
bool rows_meet_bytes(const void* a, long long as, long long aw, int T, const void* b, long long bytes) {
  const long long a0 = static_cast<long long>(reinterpret_cast<uintptr_t>(a)), b0 = static_cast<long long>(reinterpret_cast<uintptr_t>(b));
  if (a0 + 2 * ((T - 1) * as + aw) <= b0 || b0 + bytes <= a0) return false;
  if (b0 < a0) return true;
  const long long off = (b0 - a0) % (2 * as);  // behind the row before it
  return off < 2 * aw || off + bytes > 2 * as;
}

// SMs of the current device, looked up once; a GB300's where there is none.
int paged_sms() {
  const int sms = fa::device_sm_count();
  return sms > 0 ? sms : 152;
}

int paged_max_kv(const fa_paged_cache* c, const fa_paged_batch* b) {
  const long long most = static_cast<long long>(b->max_pages) * c->page_size;
  return static_cast<int>(b->max_kv > 0 && b->max_kv < most ? b->max_kv : most);
}

}  // namespace

int fa_paged_append(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* k,
                    long long k_stride, const void* v, long long v_stride, const void* q,
                    long long q_stride, void* q_out, long long q_out_stride, int Hq, const float* cos,
                    const float* sin, int max_pos, int rot, int interleaved, void* cuda_stream) {
  fa::PagedPool pool;
  fa::PagedBatchDev dev;
  bool empty = false;
  int rc = check_paged(cache, batch, &pool, &dev, &empty);
  if (rc != FA_OK) return rc;
  const int d = cache->d;
  if (Hq < 0 || rot < 0 || rot > d || max_pos < 0) return FA_ERR_INVALID;
  if (rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (empty) return FA_OK;
  if (!fa::aligned16(k) || !fa::aligned16(v) || !row_stride_ok(k_stride, pool.num_heads, d) ||
      !row_stride_ok(v_stride, pool.num_heads, d))
    return FA_ERR_INVALID;
  if (Hq > 0 && (!fa::aligned16(q) || !fa::aligned16(q_out) || !row_stride_ok(q_stride, Hq, d) ||
                 !row_stride_ok(q_out_stride, Hq, d)))
    return FA_ERR_INVALID;
  if (Hq > 0) {
    const long long qw = static_cast<long long>(Hq) * d, kw = static_cast<long long>(pool.num_heads) * d;
    const bool in_place = q_out == q && (q_out_stride == q_stride || dev.T == 1);
    if ((!in_place && rows_meet(q_out, q_out_stride, qw, q, q_stride, qw, dev.T)) ||
        rows_meet(q_out, q_out_stride, qw, k, k_stride, kw, dev.T) ||
        rows_meet(q_out, q_out_stride, qw, v, v_stride, kw, dev.T))
      return FA_ERR_INVALID;
  }
  if (rot > 0 && (!fa::aligned16(cos) || !fa::aligned16(sin) || max_pos == 0)) return FA_ERR_INVALID;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  const fa::PagedAppend p{k, v, q, q_out, k_stride, v_stride, q_stride, q_out_stride, Hq,
                          cos, sin, max_pos, rot, interleaved ? 1 : 0};
  return fa::launch_paged_append(pool, dev, p, static_cast<cudaStream_t>(cuda_stream));
}

size_t fa_paged_attn_workspace_bytes(const fa_paged_cache* cache, const fa_paged_batch* batch, int Hq) {
  fa::PagedPool pool;
  fa::PagedBatchDev dev;
  bool empty = false;
  if (check_paged(cache, batch, &pool, &dev, &empty) != FA_OK || empty || Hq <= 0 || Hq % cache->num_heads != 0)
    return 0;
  return fa::paged_attn_plan(pool, dev, Hq, paged_max_kv(cache, batch), paged_sms()).workspace_bytes;
}

int fa_paged_attn(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* q,
                  long long q_stride, void* o, float* lse, int Hq, int window, float scale,
                  void* workspace, size_t ws_bytes, void* cuda_stream) {
  fa::PagedPool pool;
  fa::PagedBatchDev dev;
  bool empty = false;
  int rc = check_paged(cache, batch, &pool, &dev, &empty);
  if (rc != FA_OK) return rc;
  if (Hq <= 0 || Hq % cache->num_heads != 0 || window < 0) return FA_ERR_INVALID;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID;
  if (empty) return FA_OK;
  if (!fa::aligned16(q) || !fa::aligned16(o) || !aligned4(lse) || !row_stride_ok(q_stride, Hq, cache->d))
    return FA_ERR_INVALID;
  // o may be q itself: a row is read before it is written, by the CTA that writes it or by a kernel before
  const long long width = static_cast<long long>(Hq) * cache->d;
  if (!(o == q && (q_stride == width || dev.T == 1)) && rows_meet(o, width, width, q, q_stride, width, dev.T))
    return FA_ERR_INVALID;
  // no length exceeds the block table's: a window as long masks nothing, and edges of shorter ones fit an int
  if (window >= static_cast<long long>(batch->max_pages) * cache->page_size) window = 0;
  // packed (query, head) rows of a key head are counted in 32 bits
  if (static_cast<long long>(batch->max_q) * Hq > 0x7fffffffLL - 4096) return FA_ERR_INVALID;
  const fa::PagedPlan plan = fa::paged_attn_plan(pool, dev, Hq, paged_max_kv(cache, batch), paged_sms());
  if (plan.workspace_bytes > 0 &&
      (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
       ws_bytes < plan.workspace_bytes))
    return FA_ERR_WORKSPACE;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  const fa::PagedAttn p{q, q_stride, o, lse, Hq, window, scale};
  return fa::launch_paged_attn(pool, dev, p, plan, workspace, static_cast<cudaStream_t>(cuda_stream));
}

namespace {

// Sizes of a packed call.
int check_packed(int B, int T, int Hq, int Hkv, int d) {
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B < 0 || T < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0) return FA_ERR_INVALID;
  if (Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;  // a tile of 128 rows holds a token's group
  // rows of a key head, items, and a token with a window behind it are counted in 32 bits
  if (static_cast<long long>(T) * Hq > 0x7fffffffLL - 4096 || T > 0x3fffffff || static_cast<long long>(B) * Hkv > 0x3fffffffLL)
    return FA_ERR_INVALID;
  return FA_OK;
}

// The kernels scale scores in units of log2.
bool packed_scale_ok(float scale) { return scale >= 0.f && std::isfinite(scale * 1.4426950408889634f); }

// row_stride_ok for rows that a tensor map names (strides below 2^40 bytes).
bool map_stride_ok(long long stride, int heads, int d) { return row_stride_ok(stride, heads, d) && stride < (1LL << 38); }

fa::PackedShape packed_shape(const int* cu, int B, int T, int Hq, int Hkv, int causal, int window) {
  // no sequence is longer than T: a window as long masks nothing
  return fa::PackedShape{cu, B, T, Hq, Hkv, 128 / (Hq / Hkv), causal ? 1 : 0, window >= T ? 0 : window,
                         fa::GroupDiv::of(Hq / Hkv), fa::GroupDiv::of(Hkv)};
}

bool workspace_ok(const void* workspace, size_t have, size_t need) {
  return need == 0 ||
         (workspace != nullptr && (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 && have >= need);
}

}  // namespace

size_t fa_packed_fwd_workspace_bytes(int B, int T, int Hq, int Hkv, int d) {
  if (check_packed(B, T, Hq, Hkv, d) != FA_OK || B == 0 || T == 0) return 0;
  return fa::packed_fwd_workspace_bytes(B, T, Hq, Hkv, d, paged_sms());
}

int fa_packed_fwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                  long long v_stride, const int* cu, int B, int T, int Hq, int Hkv, int d, int causal, int window,
                  float scale, void* o, float* lse, void* workspace, size_t ws_bytes, void* cuda_stream) {
  int rc = check_packed(B, T, Hq, Hkv, d);
  if (rc != FA_OK) return rc;
  if (!packed_scale_ok(scale) || window < 0 || (window > 0 && !causal)) return FA_ERR_INVALID;
  if (B == 0 || T == 0) return FA_OK;
  if (!fa::aligned16(q) || !fa::aligned16(k) || !fa::aligned16(v) || !fa::aligned16(o) || !aligned4(lse) ||
      !aligned4(cu) || !map_stride_ok(q_stride, Hq, d) || !map_stride_ok(k_stride, Hkv, d) ||
      !map_stride_ok(v_stride, Hkv, d))
    return FA_ERR_INVALID;
  const long long qw = static_cast<long long>(Hq) * d, kw = static_cast<long long>(Hkv) * d;
  if (rows_meet(o, qw, qw, q, q_stride, qw, T) || rows_meet(o, qw, qw, k, k_stride, kw, T) ||
      rows_meet(o, qw, qw, v, v_stride, kw, T))
    return FA_ERR_INVALID;
  if (!workspace_ok(workspace, ws_bytes, fa::packed_fwd_workspace_bytes(B, T, Hq, Hkv, d, paged_sms())))
    return FA_ERR_WORKSPACE;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  const fa::PackedProblem p{q, k, v, q_stride, k_stride, v_stride,
                            packed_shape(cu, B, T, Hq, Hkv, causal, window), d, scale};
  return fa::launch_packed_fwd(p, o, lse, workspace, static_cast<cudaStream_t>(cuda_stream));
}

size_t fa_packed_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int d) {
  if (check_packed(B, T, Hq, Hkv, d) != FA_OK || B == 0 || T == 0) return 0;
  return fa::packed_bwd_workspace_bytes(B, T, Hq, Hkv, paged_sms());
}

int fa_packed_bwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                  long long v_stride, const void* o, const float* lse, const void* dO, long long do_stride,
                  const int* cu, int B, int T, int Hq, int Hkv, int d, int causal, int window, float scale,
                  void* dq, long long dq_stride, void* dk, long long dk_stride, void* dv, long long dv_stride,
                  void* workspace, size_t ws_bytes, void* cuda_stream) {
  int rc = check_packed(B, T, Hq, Hkv, d);
  if (rc != FA_OK) return rc;
  if (!packed_scale_ok(scale) || window < 0 || (window > 0 && !causal)) return FA_ERR_INVALID;
  if (B == 0 || T == 0) return FA_OK;
  struct Rows {
    const void* at;
    long long stride;
    int heads;
  };
  const Rows in[5] = {{q, q_stride, Hq}, {k, k_stride, Hkv}, {v, v_stride, Hkv}, {dO, do_stride, Hq},
                      {o, static_cast<long long>(Hq) * d, Hq}};
  const Rows out[3] = {{dq, dq_stride, Hq}, {dk, dk_stride, Hkv}, {dv, dv_stride, Hkv}};
  for (const Rows& r : in)
    if (!fa::aligned16(r.at) || !map_stride_ok(r.stride, r.heads, d)) return FA_ERR_INVALID;
  for (const Rows& r : out)
    if (!fa::aligned16(r.at) || !row_stride_ok(r.stride, r.heads, d)) return FA_ERR_INVALID;
  if (!aligned4(lse) || !aligned4(cu)) return FA_ERR_INVALID;
  auto meet = [&](const Rows& a, const Rows& b) {
    return rows_meet(a.at, a.stride, static_cast<long long>(a.heads) * d, b.at, b.stride,
                     static_cast<long long>(b.heads) * d, T);
  };
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (meet(out[i], r)) return FA_ERR_INVALID;
    const long long width = static_cast<long long>(out[i].heads) * d;
    if (rows_meet_bytes(out[i].at, out[i].stride, width, T, lse, 4LL * T * Hq) ||
        rows_meet_bytes(out[i].at, out[i].stride, width, T, cu, 4LL * (B + 1)))
      return FA_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return FA_ERR_INVALID;
  }
  if (!workspace_ok(workspace, ws_bytes, fa::packed_bwd_workspace_bytes(B, T, Hq, Hkv, paged_sms())))
    return FA_ERR_WORKSPACE;
  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  const fa::PackedBwd b{{q, k, v, q_stride, k_stride, v_stride, packed_shape(cu, B, T, Hq, Hkv, causal, window), d, scale},
                        o, lse, dO, do_stride, dq, dk, dv, dq_stride, dk_stride, dv_stride};
  return fa::launch_packed_bwd(b, workspace, static_cast<cudaStream_t>(cuda_stream));
}

int fa_rope_axes(const void* q, long long q_stride, void* q_out, long long q_out_stride, int Hq, const void* k,
                 long long k_stride, void* k_out, long long k_out_stride, int Hk, const int* positions,
                 int num_axes, int T, const unsigned char* axis_of, const float* cos, const float* sin,
                 int max_pos, int rot, int d, int interleaved, int inverse, void* cuda_stream) {
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (Hq < 0 || Hk < 0 || T < 0 || num_axes < 1 || num_axes > 256 || rot < 0 || rot > d || max_pos < 0)
    return FA_ERR_INVALID;
  if (rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  const long long heads = static_cast<long long>(Hq) + Hk;
  if (heads > 0x7fffff) return FA_ERR_INVALID;
  if (T == 0 || heads == 0) return FA_OK;
  if (rot > 0 && (max_pos == 0 || axis_of == nullptr || !aligned4(positions) || !fa::aligned16(cos) ||
                  !fa::aligned16(sin)))
    return FA_ERR_INVALID;
  if (Hq > 0 && (!fa::aligned16(q) || !fa::aligned16(q_out) || !row_stride_ok(q_stride, Hq, d) ||
                 !row_stride_ok(q_out_stride, Hq, d)))
    return FA_ERR_INVALID;
  if (Hk > 0 && (!fa::aligned16(k) || !fa::aligned16(k_out) || !row_stride_ok(k_stride, Hk, d) ||
                 !row_stride_ok(k_out_stride, Hk, d)))
    return FA_ERR_INVALID;
  const long long qw = static_cast<long long>(Hq) * d, kw = static_cast<long long>(Hk) * d;
  if (Hq > 0 && !(q_out == q && (q_out_stride == q_stride || T == 1)) &&
      rows_meet(q_out, q_out_stride, qw, q, q_stride, qw, T))
    return FA_ERR_INVALID;
  if (Hk > 0 && !(k_out == k && (k_out_stride == k_stride || T == 1)) &&
      rows_meet(k_out, k_out_stride, kw, k, k_stride, kw, T))
    return FA_ERR_INVALID;
  if (Hq > 0 && Hk > 0 && (rows_meet(q_out, q_out_stride, qw, k, k_stride, kw, T) ||
                           rows_meet(k_out, k_out_stride, kw, q, q_stride, qw, T) ||
                           rows_meet(q_out, q_out_stride, qw, k_out, k_out_stride, kw, T)))
    return FA_ERR_INVALID;
  fa::RopeProblem p{q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, Hq, Hk, positions, cos, sin,
                    T, d, rot, max_pos, interleaved ? 1 : 0, inverse ? 1 : 0, {}};
  for (int i = 0; i < rot / 2; ++i) {
    if (axis_of[i] >= num_axes) return FA_ERR_INVALID;
    p.axes.of[i] = axis_of[i];
  }
  for (int u = 0; u < rot / 16; ++u) {
    bool whole = true;
    for (int i = 1; i < 8; ++i) whole = whole && axis_of[8 * u + i] == axis_of[8 * u];
    p.axes.whole |= whole ? 1u << u : 0u;
  }
  fa::DeviceState* st = nullptr;
  const int rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  return fa::launch_rope_axes(p, static_cast<cudaStream_t>(cuda_stream));
}

int fa_get_last_device_status(void) {
  fa::DeviceState* st = nullptr;
  if (fa::current_device(&st) != FA_OK) return FA_ERR_LAUNCH;
  if (cudaDeviceSynchronize() != cudaSuccess) return FA_ERR_LAUNCH;
  int word = 0;
  if (cudaMemcpyFromSymbol(&word, fa::g_status_word, sizeof(int)) != cudaSuccess)
    return FA_ERR_LAUNCH;
  const int zero = 0;
  if (cudaMemcpyToSymbol(fa::g_status_word, &zero, sizeof(int)) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return word == fa::kStatusTimeout ? FA_ERR_TIMEOUT : word == fa::kStatusIndex ? FA_ERR_INDEX : FA_OK;
}

}  // extern "C"
