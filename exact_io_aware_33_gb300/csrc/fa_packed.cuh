// What the kernels of packed attention share: the batch and its bounds checks,
// the tiles of a sequence, and how work is found.
//
// Rows are packed twice. Tokens of all sequences lie one after another (cu
// marks where each begins), and the G query heads that read a key head share
// its tiles: a tile of query rows holds `tpt` = floor(128 / G) tokens with
// their G heads each, token by token, so row r of a tile is token r / G, head r
// % G of the group. One box of a 4-D tensor map fetches it: extents (64
// channels, G, 1, tpt) of [T, Hkv, G, d]. Short sequences fill their tiles G
// times as well as with a head per tile, a causal tile has 128 / G positions'
// spread, and the gradients of a shared key head are summed in its own
// accumulator, in a fixed order.
//
// Everything the device reads as an index (cu) is checked against the sizes
// that the host gave before it is used: what fails is clamped and kStatusIndex
// is raised, so a bad table never becomes a bad address. Nor endless work: a list
// of borders that fall somewhere stays empty (sequences that overlap could have any
// number of rows).
#pragma once

#include <cuda_bf16.h>

#include "fa_paged.cuh"

namespace fa {

constexpr int kKeyTile = 128;

// What the kernels read of the borders and lists they take from L2: the dQ kernel
// reads what was written before the kernel ahead of it, which alone has waited.
// (make_list, after a wait of its own, reads the borders twice, and may cache them.)

// Sum of x over this lane and those before it.
__device__ __forceinline__ int warp_prefix(int x, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// First row of sequence b and its number of rows.
struct PackedSeq {
  int row0, n;
  bool fell;  // ends before it begins
};

template <bool kCache = false>
__device__ __forceinline__ PackedSeq packed_seq(const PackedShape& s, int b, int* status) {
  const int c0 = kCache ? s.cu[b] : __ldcg(s.cu + b), c1 = kCache ? s.cu[b + 1] : __ldcg(s.cu + b + 1);
  PackedSeq q;
  q.row0 = min(max(c0, 0), s.T);
  q.n = min(max(c1, q.row0), s.T) - q.row0;
  q.fell = c1 < c0;
  if (c0 < 0 || c1 < c0 || c1 > s.T) raise_index(status);
  return q;
}

// Key tiles [lo, lo + n) that the tokens [i0, i1) of a sequence of `len` see (none when i0 >= i1).
struct TileRange {
  int lo, n;
};
__device__ __forceinline__ TileRange keys_of(const PackedShape& s, int len, int i0, int i1) {
  const int end = s.causal ? i1 : len;
  const int lo = s.window > 0 ? max(i0 - s.window + 1, 0) / kKeyTile : 0;
  return TileRange{lo, i0 < i1 ? (end + kKeyTile - 1) / kKeyTile - lo : 0};
}

// Tiles of query rows [lo, lo + n) that see some of the keys [k0, k1) of a sequence of `len`.
__device__ __forceinline__ TileRange rows_of(const PackedShape& s, int len, int k0, int k1) {
  const int end = s.window > 0 ? min(len, k1 - 1 + s.window) : len;
  const int lo = s.causal ? k0 / s.tpt : 0;
  return TileRange{lo, k0 < k1 ? (end + s.tpt - 1) / s.tpt - lo : 0};
}

// An entry of the work: `unit` tokens of a sequence from token i0 on. With a
// key head it is an item.
struct PackedEntry {
  int row0, n, i0;
};

// Entry number e when the sequences' entries are laid end to end, found by a
// whole warp; n = 0 when there are fewer.
__device__ __forceinline__ PackedEntry find_entry(const PackedShape& s, const PackedList& l, int e, int* status) {
  const int lane = static_cast<int>(lane_id());
  int before = 0;
  for (int b0 = 0; b0 < s.B; b0 += 32) {
    PackedSeq q{0, 0, false};
    if (b0 + lane < s.B) q = packed_seq(s, b0 + lane, status);
    const int own = q.n < l.least ? 0 : (q.n + l.unit - 1) / l.unit;
    const int end = warp_prefix(own, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, before + end > e);
    if (past) {
      const int src = __ffs(past) - 1;
      const int first = before + __shfl_sync(0xffffffffu, end - own, src);
      return PackedEntry{__shfl_sync(0xffffffffu, q.row0, src), __shfl_sync(0xffffffffu, q.n, src), (e - first) * l.unit};
    }
    before += __shfl_sync(0xffffffffu, end, 31);
  }
  return PackedEntry{0, 0, 0};
}

// Hands out items: the CTA's own one where every item has a CTA (no list), or
// the list's, heaviest first, by a counter. The next item's number is asked for
// kAhead steps before the loads of the present one end, so that the answer is
// not waited for; sooner would deal items out before it is known who is done
// first (a whole item sooner: 191 us instead of 181 to 189 for 8192 causal rows, 16
// heads, d = 128).
struct ItemQueue {
  static constexpr int kAhead = 4;
  const PackedList* list;
  GroupDiv by_head;
  int count;  // entries
  int next;   // number of the next item; -1: not asked for
  PackedEntry own;

  // By the whole warp.
  __device__ __forceinline__ void start(const PackedShape& s, const PackedList& l, int* status) {
    list = &l;
    by_head = s.by_head;
    next = static_cast<int>(blockIdx.x);
    if (l.entries == nullptr)
      own = find_entry(s, l, by_head.div(next), status);
    else
      count = __ldcg(&l.head->count);
  }
  // By lane 0, with `left` steps of the present item still to be loaded, this one included.
  __device__ __forceinline__ void step(int left) {
    if (next < 0 && left <= kAhead)
      next = list->entries == nullptr ? 0x7fffffff
                                      : static_cast<int>(gridDim.x) + atomicAdd(&list->head->taken, 1);
  }
  // The next item, for lane 0; false when there are no more.
  __device__ __forceinline__ bool take(PackedEntry* e, int* h) {
    const int k = by_head.div(next);
    if (list->entries == nullptr) {
      if (next == 0x7fffffff || own.n == 0) return false;
      *e = own;
    } else {
      if (k >= count) return false;
      const int4 r = __ldcg(list->entries + k);
      *e = PackedEntry{r.x, r.y, r.z};
    }
    *h = next - k * by_head.G;
    next = -1;
    return true;
  }
};

// ---------------------------------------------------------------- the order of the work
// Sequences of different lengths give items whose costs differ by orders of
// magnitude, so they are handed out heaviest first: each CTA takes the next one
// when it is done with its last, and the light ones even out the ends. One
// block sorts the entries (tokens of a sequence; each key head makes an item of
// it) by their cost in steps: a counting sort with a bucket per step. The
// order within a bucket is left to chance; no result depends on it, since an
// item's result does not depend on who computes it.
constexpr int kBuckets = 1024;  // costs from here up share one: beyond 1023 steps the order is left to chance, too

__device__ __forceinline__ int cost_of(const PackedShape& s, const PackedList& l, int n, int i0) {
  const int i1 = min(i0 + l.unit, n);
  return l.keys ? rows_of(s, n, i0, i1).n : keys_of(s, n, i0, i1).n;
}

// Makes list l, by a block of kThreads. Where borders rise, its entries are no
// more than l.cap = T / l.unit + B.
template <int kThreads>
__device__ __forceinline__ void make_list(const PackedShape& s, const PackedList& l, int* status) {
  constexpr int kWarps = kThreads / 32, kOwn = kBuckets / kThreads;  // buckets per thread, when their beginnings are summed up
  static_assert(kBuckets % kThreads == 0, "buckets are divided evenly");
  __shared__ int bucket[kBuckets];  // heaviest first
  __shared__ int sums[32];
  __shared__ int bad;  // borders fall
  const int tid = threadIdx.x, warp = warp_id(), lane = static_cast<int>(lane_id());
  for (int i = 0; i < kOwn; ++i) bucket[tid + i * kThreads] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  // Few sequences: a warp takes one at a time, its lanes the entries. Many: it
  // takes up to 32 neighbours at a time, and its lanes their entries end to end
  // (4096 sequences of up to 16 tokens, 8 / 2 heads, d = 128: 170 us instead of 273,
  // backward 294 instead of 472; few would pay for the search).
  const int per = min(s.B / kWarps, 32);
  auto each = [&](auto&& f) {
    auto entry = [&](const PackedSeq& q, int i) { f(q, i, kBuckets - 1 - min(cost_of(s, l, q.n, i), kBuckets - 1)); };
    if (per <= 1) {  // (two sequences a warp at most)
      for (int b = warp; b < s.B; b += kWarps) {
        const PackedSeq q = packed_seq<true>(s, b, status);
        if (q.fell) bad = 1;
        if (q.n < l.least) continue;
        for (long long i0 = static_cast<long long>(lane) * l.unit; i0 < q.n; i0 += 32LL * l.unit)
          entry(q, static_cast<int>(i0));
      }
      return;
    }
    int seen = 0;  // entries of this warp so far
    for (int b0 = warp * per; b0 < s.B; b0 += kWarps * per) {
      PackedSeq q{0, 0, false};
      if (lane < per && b0 + lane < s.B) q = packed_seq<true>(s, b0 + lane, status);
      const int own = q.n < l.least ? 0 : (q.n + l.unit - 1) / l.unit;
      const int end = warp_prefix(own, lane), total = __shfl_sync(0xffffffffu, end, 31);
      if (__any_sync(0xffffffffu, q.fell) || total > l.cap - seen) {
        bad = 1;
        return;
      }
      seen += total;
      for (int e0 = 0; e0 < total; e0 += 32) {
        const int e = e0 + lane;
        int src = 0;  // its sequence: as many of them end before it
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
          if (__shfl_sync(0xffffffffu, end, src + m - 1) <= e) src += m;
        const PackedSeq of{__shfl_sync(0xffffffffu, q.row0, src), __shfl_sync(0xffffffffu, q.n, src), false};
        const int i = (e - __shfl_sync(0xffffffffu, end - own, src)) * l.unit;
        if (e < total) entry(of, i);
      }
    }
  };
  each([&](const PackedSeq&, int, int k) { atomicAdd(&bucket[k], 1); });
  __syncthreads();
  // where each bucket begins
  int own[kOwn], all = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) all += own[i] = bucket[tid * kOwn + i];
  const int end = warp_prefix(all, lane);
  if (lane == 31) sums[warp] = end;
  __syncthreads();
  int before = end - all + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    bucket[tid * kOwn + i] = before;
    before += own[i];
  }
  if (tid == kThreads - 1) *l.head = PackedHead{bad ? 0 : before, 0, {}};
  __syncthreads();
  if (bad) return;
  each([&](const PackedSeq& q, int i, int k) {
    const int at = atomicAdd(&bucket[k], 1);
    if (at < l.cap) l.entries[at] = make_int4(q.row0, q.n, i, 0);
  });
}

// Zeroes rows [row, rows) of a tile of `chunks` 128-byte-swizzled chunks, thread `tid` of `threads`.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int chunk_bytes, int chunks, int row, int rows, int tid,
                                          int threads) {
  uint8_t* at = tile + (tid & 7) * 16;
#pragma unroll 2
  for (int r = row + tid / 8; r < rows; r += threads / 8)
#pragma unroll
    for (int c = 0; c < chunks; ++c) *reinterpret_cast<uint4*>(at + c * chunk_bytes + r * 128) = make_uint4(0, 0, 0, 0);
}

}  // namespace fa
