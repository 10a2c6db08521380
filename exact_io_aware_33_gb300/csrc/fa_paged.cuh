// What the kernels of the paged 8-bit key/value cache share: the packed
// batch, its bounds checks, and e4m3 conversions.
//
// Pool layout: k_pages and v_pages are e4m3 [num_pages, heads, page_size, d],
// so the tokens of one head in one page are one contiguous block (1 to 16
// KiB) that a tiled copy fetches whole; k_scales and v_scales are fp32
// [num_pages, heads]. A cached value is code * scale.
//
// Everything the device reads as an index (block_table, kv_lens, cu_q) is
// checked against the sizes the host gave before it is used; what fails the
// check is treated as absent and kStatusIndex is raised, so a bad table never
// becomes a bad address.
//
// Launch overlap. The attention's streaming and chunk kernels need every SM
// for themselves: one that starts while its predecessor's blocks are still
// there places fewer of its CTAs on some SMs and keeps them so for the whole
// run (8 sequences of 8192 keys, 32 heads, one call after another: 119 us,
// 87 us otherwise). So the kernels that come before it in a step, the append
// and the joins, do not call grid_dep_launch: the next kernel is launched
// ahead and starts when their last block ends, which is still some 3 us
// sooner than without programmatic serialization.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// An index was out of range. A timeout that the status word already holds
// stays: it says more, that results are missing.
__device__ __forceinline__ void raise_index(int* status) { atomicCAS(status, kStatusOk, kStatusIndex); }

// One sequence of the batch: its packed rows [row0, row0 + n) and its length.
struct PagedSeq {
  int row0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatchDev& b, int seq, int* status) {
  PagedSeq s;
  bool bad = false;
  if (b.cu_q != nullptr) {
    const int c0 = b.cu_q[seq], c1 = b.cu_q[seq + 1];
    bad = c0 < 0 || c1 < c0 || c1 > b.T || c1 - c0 > b.max_q;
    s.row0 = min(max(c0, 0), b.T);
    s.n = min(min(max(c1, s.row0), b.T) - s.row0, b.max_q);
  } else {
    s.row0 = seq;
    s.n = 1;
  }
  s.len = b.kv_lens[seq];
  // max_pages * page_size fits an int: checked on the host
  const int most = b.max_pages << b.page_shift;
  bad = bad || s.len < 0 || s.len > most;
  s.len = min(max(s.len, 0), most);
  if (bad) raise_index(status);
  return s;
}

// The page that holds the tokens [idx * page_size, ...) of a sequence, or -1.
__device__ __forceinline__ int paged_page(const PagedBatchDev& b, int seq, int idx, int* status) {
  const int p = b.block_table[static_cast<long long>(seq) * b.max_pages + idx];
  if (p >= 0 && p < b.num_pages) return p;
  raise_index(status);
  return -1;
}

// r / G for a packed row 0 <= r < 2^31 without a division: with m = floor(2^32
// / G), r m / 2^32 is less than r / 2^32 < 1 below r / G, so its floor is the
// quotient or one less, and the remainder tells which.
struct GroupDiv {
  int G;
  uint32_t magic;
  __host__ static GroupDiv of(int g) {
    return GroupDiv{g, g == 1 ? 0xffffffffu : static_cast<uint32_t>((1ull << 32) / static_cast<unsigned>(g))};
  }
  __device__ __forceinline__ int div(int r) const {
    int q = static_cast<int>(__umulhi(static_cast<uint32_t>(r), magic));
    if (r - q * G >= G) ++q;
    return q;
  }
};

// Left in the workspace by each part of a divided launch, for the kernel that
// joins the pieces of items: the item that the part begins and does not end.
struct JoinRecord {
  int parts;      // that hold a piece of it, this one first; 0: there is no such item
  int row0;       // first token row of its sequence
  int h;          // key head
  int r0, rows;   // its first packed row, and the sequence's packed rows
  int pad[3];
};

// Parts that hold units before `end` from part c on, of `parts` equal parts of
// `units`: part k starts at floor(k units / parts), which is below `end` for k
// < end parts / units.
__device__ __forceinline__ int parts_until(long long end, long long units, int parts, int c) {
  return static_cast<int>((end * parts + units - 1) / units) - c;
}

// Two e4m3 codes (low byte first) to an f16 pair; exact, and a NaN code gives NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// Two floats to two e4m3 codes, to nearest even, magnitudes above 448 to 448; `lo` in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 0xff in each byte of w that holds a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t z = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (z >> 7) * 255u;
}

// The first key that the query at position p sees. Before position 0 (rows of
// a padded batch) it sees none, and p - window may lie below the int range.
__device__ __forceinline__ int first_seen(int p, int window) {
  return window > 0 ? max(max(p, 0) - window + 1, 0) : 0;
}

// Whether the query at position p sees key j. (p - window is formed for p >= j >= 0 only.)
__device__ __forceinline__ bool sees(int p, int j, int window) {
  return j <= p && (window == 0 || j > p - window);
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace fa
