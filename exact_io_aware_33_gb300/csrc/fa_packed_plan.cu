// The order of the work of a packed attention call.
//
// Sequences of different lengths give items whose costs differ by orders of
// magnitude, so they are handed out heaviest first: each CTA takes the next one
// when it is done with its last, and the light ones even out the ends. One
// block sorts the entries (tokens of a sequence; each key head makes an item of
// it) by their cost in steps: a counting sort with a bucket per step, a warp
// per sequence. The order within a bucket is left to chance; no result depends
// on it, since an item's result does not depend on who computes it.
//
// Bound by latency: 3 us for 8 sequences of 4096 tokens (256 entries).

#include "fa_packed.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = 1024;  // costs from here up share one

struct PlanArgs {
  PackedShape s;
  PackedList lists[2];
  int* status;
};

__device__ __forceinline__ int cost_of(const PackedShape& s, const PackedList& l, int n, int i0) {
  const int i1 = min(i0 + l.unit, n);
  return l.keys ? rows_of(s, n, i0, i1).n : keys_of(s, n, i0, i1).n;
}

__global__ void __launch_bounds__(kThreads, 1) packed_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int bucket[kBuckets];  // heaviest first
  __shared__ int sums[32];
  const PackedList& l = a.lists[blockIdx.x];
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  bucket[tid] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  auto each = [&](auto&& f) {
    for (int b = warp; b < a.s.B; b += kThreads / 32) {
      const PackedSeq q = packed_seq(a.s, b, a.status);
      for (long long i0 = static_cast<long long>(lane) * l.unit; i0 < q.n; i0 += 32LL * l.unit) {
        const int i = static_cast<int>(i0);
        f(q, i, kBuckets - 1 - min(cost_of(a.s, l, q.n, i), kBuckets - 1));
      }
    }
  };
  each([&](const PackedSeq&, int, int k) { atomicAdd(&bucket[k], 1); });
  __syncthreads();
  // where each bucket begins
  const int own = bucket[tid];
  int end = own;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, end, m);
    if (lane >= m) end += x;
  }
  if (lane == 31) sums[warp] = end;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += sums[w];
  bucket[tid] = before + end - own;
  if (tid == kThreads - 1) {
    // (sequences that overlap could be more than there is room for)
    if (before + end > l.cap) raise_index(a.status);
    *l.head = PackedHead{min(before + end, l.cap), 0, {}};
  }
  __syncthreads();
  each([&](const PackedSeq& q, int i, int k) {
    const int at = atomicAdd(&bucket[k], 1);
    if (at < l.cap) l.entries[at] = make_int4(q.row0, q.n, i, 0);
  });
}

}  // namespace

int launch_packed_plan(const PackedShape& s, const PackedList* lists, int n, cudaStream_t stream) {
  PlanArgs a{};
  a.s = s;
  a.status = device_status_word();
  if (!a.status) return -3;
  int blocks = 0;
  for (int i = 0; i < n; ++i)
    if (lists[i].entries != nullptr) a.lists[blocks++] = lists[i];
  if (blocks == 0) return 0;
  const cudaError_t e = launch_overlapped(packed_plan_kernel, dim3(blocks), dim3(kThreads), 0, stream, a);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace fa
