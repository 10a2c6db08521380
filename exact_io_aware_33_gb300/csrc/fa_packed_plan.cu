// The order of the work of a packed attention call.
//
// Sequences of different lengths give items whose costs differ by orders of
// magnitude, so they are handed out heaviest first: each CTA takes the next one
// when it is done with its last, and the light ones even out the ends. One
// block sorts the entries (tokens of a sequence; each key head makes an item of
// it) by their cost in steps: a counting sort with a bucket per step. The
// order within a bucket is left to chance; no result depends on it, since an
// item's result does not depend on who computes it.
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
  // Few sequences: a warp takes one at a time, its lanes the entries. Many: it
  // takes up to 32 neighbours at a time, and its lanes their entries end to end
  // (4096 sequences of up to 16 tokens: 125 us less; 8 of up to 4096: 2 us more,
  // for the search).
  const int per = min(a.s.B / (kThreads / 32), 32);
  auto each = [&](auto&& f) {
    auto entry = [&](const PackedSeq& q, int i) { f(q, i, kBuckets - 1 - min(cost_of(a.s, l, q.n, i), kBuckets - 1)); };
    if (per <= 1) {
      for (int b = warp; b < a.s.B; b += kThreads / 32) {
        const PackedSeq q = packed_seq(a.s, b, a.status);
        for (long long i0 = static_cast<long long>(lane) * l.unit; i0 < q.n; i0 += 32LL * l.unit)
          entry(q, static_cast<int>(i0));
      }
      return;
    }
    for (int b0 = warp * per; b0 < a.s.B; b0 += kThreads / 32 * per) {
      PackedSeq q{0, 0};
      if (lane < per && b0 + lane < a.s.B) q = packed_seq(a.s, b0 + lane, a.status);
      const int own = (q.n + l.unit - 1) / l.unit;
      const int end = warp_prefix(own, lane), total = __shfl_sync(0xffffffffu, end, 31);
      for (int e0 = 0; e0 < total; e0 += 32) {
        const int e = e0 + lane;
        int src = 0;  // its sequence: as many of them end before it
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
          if (__shfl_sync(0xffffffffu, end, src + m - 1) <= e) src += m;
        const PackedSeq of{__shfl_sync(0xffffffffu, q.row0, src), __shfl_sync(0xffffffffu, q.n, src)};
        const int i = (e - __shfl_sync(0xffffffffu, end - own, src)) * l.unit;
        if (e < total) entry(of, i);
      }
    }
  };
  each([&](const PackedSeq&, int, int k) { atomicAdd(&bucket[k], 1); });
  __syncthreads();
  // where each bucket begins
  const int own = bucket[tid];
  const int end = warp_prefix(own, lane);
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
