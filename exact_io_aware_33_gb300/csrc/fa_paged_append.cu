// Appending rotated keys and values to a paged e4m3 cache.
//
// Mathematics. Token i of sequence b sits at position p = kv_lens[b] - n_b + i.
// Its key (and its query) is rotated: each channel pair (a, b) of the first
// `rot` channels becomes (a cos - b sin, b cos + a sin) with the angle tables'
// row p; pairs are (c, c + rot/2), or (2c, 2c + 1) when interleaved. Products
// and sums are rounded one by one in fp32 (no fused multiply-add), so that a
// key's code does not depend on which kernel rotated it.
// A page and head share one power-of-two scale s for keys and one for values:
//   s_new = smallest power of two with max |x| / s <= 448 over the new tokens,
//   s     = s_new for a page that the call begins, else max(s_old, s_new),
//   code  = e4m3(x / s).
// Powers of two make x / s exact, so a code carries one rounding, and when a
// page's scale grows its older codes are multiplied by s_old / s, which is
// exact too until they fall below e4m3's normal range, where they are rounded
// once more. Values that are not finite do not take part in the maximum; an
// infinity is stored as 448 s, a NaN as NaN.
//
// Both kernels are bound by memory: per token they read 2 d (2 Hkv + Hq) bytes
// of bf16 and 4 rot bytes of table, and write 2 d Hkv bytes of codes and
// 2 d Hq of queries.

#include <cfloat>

#include "fa_paged.cuh"

namespace fa {
namespace {

struct AppendArgs {
  PagedBatchDev batch;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  long long k_stride, v_stride, q_stride, q_out_stride;  // elements from one token to the next
  uint8_t* k_pages;
  uint8_t* v_pages;
  float* k_scales;
  float* v_scales;
  const float* cos;
  const float* sin;
  int* status;
  int Hq, Hkv;
  int rot, max_pos;
  int interleaved;
  int page_slots;   // pages kernel: blocks along a sequence's pages (0: found by search)
  int kv_parts, q_parts;  // pages kernel: blocks per page for keys and values, and for queries
};

// 16 channels of one token and head: two runs of eight. In the rotated range
// of the half-split form run 1 lies rot/2 channels after run 0, so that both
// members of each pair are in one thread; elsewhere the runs are adjacent.
struct Unit {
  int c0, c1;
  int tab;     // index into the angle tables' row, or -1: not rotated
};

__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int u) {
  Unit r;
  if (u * 16 >= a.rot) {
    r.c0 = u * 16;
    r.c1 = r.c0 + 8;
    r.tab = -1;
  } else if (a.interleaved) {
    r.c0 = u * 16;
    r.c1 = r.c0 + 8;
    r.tab = u * 8;
  } else {
    r.c0 = u * 8;
    r.c1 = r.c0 + a.rot / 2;
    r.tab = u * 8;
  }
  return r;
}

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void load_unit(const __nv_bfloat16* row, const Unit& u, float (&x)[16]) {
  unpack8(*reinterpret_cast<const uint4*>(row + u.c0), x);
  unpack8(*reinterpret_cast<const uint4*>(row + u.c1), x + 8);
}

__device__ __forceinline__ void load_angles(const AppendArgs& a, const Unit& u, int pos, float (&c)[8],
                                            float (&s)[8]) {
  if (u.tab < 0) return;
  if (pos >= a.max_pos) {
    raise_index(a.status);
    pos = a.max_pos - 1;
  }
  const long long at = static_cast<long long>(pos) * (a.rot / 2) + u.tab;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + at));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(a.cos + at + 4));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.sin + at));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(a.sin + at + 4));
  c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
  s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

__device__ __forceinline__ void rotate(const AppendArgs& a, const Unit& u, const float (&c)[8],
                                       const float (&s)[8], float (&x)[16]) {
  if (u.tab < 0) return;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[i], x[i + 8], c[i], s[i]);
  }
}

__device__ __forceinline__ float amax16(const float (&x)[16], float m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x[i]);
    m = v <= FLT_MAX ? fmaxf(m, v) : m;
  }
  return m;
}

// The largest of a warp's non-negative values: their bits order as the values do.
__device__ __forceinline__ float warp_amax(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// Smallest power of two s (not below 2^-126) with amax / s <= 448 = 1.75 * 2^8; 1 for amax = 0.
__device__ __forceinline__ float scale_of(float amax) {
  if (amax == 0.f) return 1.f;
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.f * 2^e: up to 1.75 (fraction field 0x600000) e - 8 serves, above it e - 7
  int e = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return pow2i(max(e, -126));
}

__device__ __forceinline__ uint2 pack_e4m3(const float* x, float inv) {
  uint2 r;
  r.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  r.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* row, const Unit& u, const float (&x)[16], float inv) {
  *reinterpret_cast<uint2*>(row + u.c0) = pack_e4m3(x, inv);
  *reinterpret_cast<uint2*>(row + u.c1) = pack_e4m3(x + 8, inv);
}

__device__ __forceinline__ void store_query(__nv_bfloat16* row, const Unit& u, const float (&x)[16]) {
  *reinterpret_cast<uint4*>(row + u.c0) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  *reinterpret_cast<uint4*>(row + u.c1) = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]),
                                                     pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
}

// Eight codes times `ratio`, rounded again.
__device__ __forceinline__ uint2 rescale_codes(uint2 w, float ratio) {
  const uint32_t in[2] = {w.x, w.y};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(in[i] >> (16 * h)));
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f));
      r |= f32x2_to_e4m3x2(x.x * ratio, x.y * ratio) << (16 * h);
    }
    out[i] = r;
  }
  return make_uint2(out[0], out[1]);
}

// ---------------------------------------------------------------- one token per sequence
// A warp writes one token's key and value of one head: D/16 lanes hold the
// key, the next D/16 the value, and the maximum is taken within each group;
// when the token makes the page's scale grow, the whole warp rounds the
// page's older codes again. Further warps of the sequence rotate 512/D
// query heads each. Latency is what counts here: one dependent chain
// length -> page -> scale, no shared memory, one launch. 2.3 us for one
// sequence, 3.2 us for 256 (32 query and 8 key heads, d = 128).
template <int D>
__global__ void __launch_bounds__(128) append_one_kernel(const AppendArgs a) {
  constexpr int kUnits = D / 16;
  constexpr int kHeadsPerWarp = 32 / kUnits;  // of queries
  grid_dep_wait();  // (no early launch of the next kernel: see fa_paged.cuh)
  const int per_seq = a.Hkv + (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int seq = static_cast<int>(w / per_seq);
  if (seq >= a.batch.B) return;
  const int task = static_cast<int>(w % per_seq);
  const int lane = threadIdx.x & 31;
  const PagedSeq s = paged_seq(a.batch, seq, a.status);
  const int pos = s.len - 1;
  if (s.n < 1 || pos < 0) return;
  const Unit u = unit_of(a, lane % kUnits);
  float x[16], c[8], sn[8];
  if (task >= a.Hkv) {
    const int h = (task - a.Hkv) * kHeadsPerWarp + lane / kUnits;
    if (h >= a.Hq) return;
    load_unit(a.q + s.row0 * a.q_stride + h * D, u, x);
    load_angles(a, u, pos, c, sn);
    rotate(a, u, c, sn, x);
    store_query(a.q_out + s.row0 * a.q_out_stride + h * D, u, x);
    return;
  }
  const int kind = lane / kUnits;  // 0: key, 1: value, others idle
  const int page = paged_page(a.batch, seq, pos >> a.batch.page_shift, a.status);
  if (page < 0) return;
  const int slot = pos & (a.batch.page_size - 1);
  const long long ph = static_cast<long long>(page) * a.Hkv + task;
  float* scales = kind == 0 ? a.k_scales : a.v_scales;
  float amax = 0.f, old = 0.f;
  if (kind < 2) {
    const __nv_bfloat16* row =
        kind == 0 ? a.k + s.row0 * a.k_stride + task * D : a.v + s.row0 * a.v_stride + task * D;
    load_unit(row, u, x);
    if (slot > 0) old = scales[ph];
    if (kind == 0) {
      load_angles(a, u, pos, c, sn);
      rotate(a, u, c, sn, x);
    }
    amax = amax16(x, 0.f);
  }
#pragma unroll
  for (int m = 1; m < kUnits; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  float scale = scale_of(amax);
  if (slot > 0) scale = fmaxf(scale, old);
#pragma unroll
  for (int kd = 0; kd < 2; ++kd) {
    const float s_new = __shfl_sync(0xffffffffu, scale, kd * kUnits);
    const float s_old = __shfl_sync(0xffffffffu, old, kd * kUnits);
    if (slot > 0 && s_new > s_old) {
      uint8_t* block = (kd == 0 ? a.k_pages : a.v_pages) + ph * a.batch.page_size * D;
      const float ratio = s_old / s_new;
      for (int i = lane; i < slot * D / 8; i += 32) {
        uint2* at = reinterpret_cast<uint2*>(block) + i;
        *at = rescale_codes(*at, ratio);
      }
    }
  }
  if (kind < 2) {
    uint8_t* block = (kind == 0 ? a.k_pages : a.v_pages) + (ph * a.batch.page_size + slot) * D;
    store_codes(block, u, x, 1.f / scale);
    if (lane % kUnits == 0) scales[ph] = scale;
  }
}

// ---------------------------------------------------------------- any number of tokens
// A block takes one page of one sequence and some of its heads, a thread 16
// channels of one slot: the page's new tokens stay in registers between the
// maximum and the codes, so keys and values are read once, and a thread's
// angles are loaded once for all the heads it goes through. The next head's
// rows are fetched before the present head's maximum is waited for. Key/value
// blocks and query blocks are blocks of one launch. 64 registers per thread,
// so that an SM holds 1024 threads and some 64 KiB of rows in flight; with one
// block of 512 threads and no fetching ahead, a prompt of 8192 tokens (32
// query and 8 key heads, d = 128) took 53 us, now 38 us: 4.9 TB/s.
// Chosen on that prompt (other numbers: 39 to 41 us). 16 ragged chunks of up to
// 700 tokens, 12 heads, d = 64, pages of 16, are 2520 blocks of 64 threads, just
// more than are resident at once (16 per SM), so that call is one chain of
// length -> page -> rows and then two key heads or four rounds of queries one
// after the other: 10.7 us, 2.1 times its bytes.
constexpr int kHeadsPerBlock = 2;    // key/value heads per block
constexpr int kQHeadsPerBlock = 8;   // query heads per block

struct RawUnit {
  uint4 a, b;
};

__device__ __forceinline__ RawUnit load_raw(const __nv_bfloat16* row, const Unit& u) {
  return RawUnit{*reinterpret_cast<const uint4*>(row + u.c0), *reinterpret_cast<const uint4*>(row + u.c1)};
}
__device__ __forceinline__ void unpack(const RawUnit& r, float (&x)[16]) {
  unpack8(r.a, x);
  unpack8(r.b, x + 8);
}

template <int D>
__global__ void __launch_bounds__(1024) append_pages_kernel(const AppendArgs a) {
  constexpr int kUnits = D / 16;
  __shared__ float red[2][2][32];  // [parity of the head][key or value][warp]
  grid_dep_wait();  // (no early launch of the next kernel: see fa_paged.cuh)
  const int parts = a.kv_parts + a.q_parts;
  const long long item = blockIdx.x / parts;
  const int part = static_cast<int>(blockIdx.x % parts);
  const int ps = a.batch.page_size, shift = a.batch.page_shift;
  int seq, j;
  if (a.page_slots > 0) {
    seq = static_cast<int>(item / a.page_slots);
    j = static_cast<int>(item % a.page_slots);
  } else {
    // sequence b owns the items from floor(cu[b] / page) + 2 b on: at least as
    // many as pages its tokens can touch. Counting the sequences that begin at
    // or before this item finds it.
    int count = 0;
    for (int b0 = 0; b0 < a.batch.B; b0 += 32) {
      const int b = b0 + (threadIdx.x & 31);
      const bool before =
          b < a.batch.B && (static_cast<long long>(max(a.batch.cu_q[b], 0)) >> shift) + 2LL * b <= item;
      const int got = __popc(__ballot_sync(0xffffffffu, before));
      count += got;
      if (got < 32) break;
    }
    seq = count - 1;
    if (seq < 0) return;
    j = static_cast<int>(item - (static_cast<long long>(max(a.batch.cu_q[seq], 0)) >> shift) - 2LL * seq);
  }
  const PagedSeq s = paged_seq(a.batch, seq, a.status);
  const int old_len = s.len - s.n;                  // negative: the first tokens have no position
  const int first = max(old_len, 0);                // first new position
  const int page_idx = (first >> shift) + j;
  if ((static_cast<long long>(page_idx) << shift) >= s.len) return;  // past the end: nothing to do
  const int p0 = page_idx << shift;
  const int lo = max(first, p0), hi = min(p0 + ps, s.len);  // new positions in this page
  if (lo >= hi) return;                             // a sequence without new tokens
  const int tid = threadIdx.x, threads = blockDim.x;  // ps * kUnits of them

  const int slot = tid / kUnits;
  const Unit u = unit_of(a, tid % kUnits);
  const bool on = p0 + slot >= lo && p0 + slot < hi;
  float c[8], sn[8];
  // packed row of the token at position p: row0 + p - old_len
  const long long row = static_cast<long long>(s.row0) + p0 + slot - old_len;

  if (part >= a.kv_parts) {
    if (!on) return;
    const int h0 = (part - a.kv_parts) * kQHeadsPerBlock, h1 = min(h0 + kQHeadsPerBlock, a.Hq);
    const __nv_bfloat16* src = a.q + row * a.q_stride;
    __nv_bfloat16* dst = a.q_out + row * a.q_out_stride;
    load_angles(a, u, p0 + slot, c, sn);
    for (int h = h0; h < h1; h += 2) {  // two heads in flight (four: 42 us instead of 38)
      RawUnit w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (h + i < h1) w[i] = load_raw(src + (h + i) * D, u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (h + i >= h1) break;
        float x[16];
        unpack(w[i], x);
        rotate(a, u, c, sn, x);
        store_query(dst + (h + i) * D, u, x);
      }
    }
    return;
  }

  const int page = paged_page(a.batch, seq, page_idx, a.status);
  if (page < 0) return;
  const int held = lo - p0;  // tokens that the page held before this call
  const int h0 = part * kHeadsPerBlock, h1 = min(h0 + kHeadsPerBlock, a.Hkv);
  const __nv_bfloat16* k_src = a.k + row * a.k_stride;
  const __nv_bfloat16* v_src = a.v + row * a.v_stride;
  RawUnit next_k{}, next_v{};
  if (on) {
    next_k = load_raw(k_src + h0 * D, u);
    next_v = load_raw(v_src + h0 * D, u);
    load_angles(a, u, p0 + slot, c, sn);
  }
  for (int h = h0; h < h1; ++h) {
    const long long ph = static_cast<long long>(page) * a.Hkv + h;
    const RawUnit wk = next_k, wv = next_v;
    if (on && h + 1 < h1) {
      next_k = load_raw(k_src + (h + 1) * D, u);
      next_v = load_raw(v_src + (h + 1) * D, u);
    }
    float xk[16], mk = 0.f, mv = 0.f;
    unpack(wk, xk);
    if (on) {
      rotate(a, u, c, sn, xk);
      mk = amax16(xk, mk);
      float xv[16];
      unpack(wv, xv);
      mv = amax16(xv, mv);
    }
    mk = warp_amax(mk);
    mv = warp_amax(mv);
    float (&r)[2][32] = red[h & 1];  // two sets: the next head's writes need no second barrier
    if ((tid & 31) == 0) {
      r[0][tid >> 5] = mk;
      r[1][tid >> 5] = mv;
    }
    float k_old = 0.f, v_old = 0.f;
    if (held > 0) {
      k_old = a.k_scales[ph];
      v_old = a.v_scales[ph];
    }
    __syncthreads();
    const int w = min(tid & 31, (threads >> 5) - 1);
    mk = warp_amax(r[0][w]);
    mv = warp_amax(r[1][w]);
    const float k_scale = fmaxf(scale_of(mk), k_old), v_scale = fmaxf(scale_of(mv), v_old);
    uint8_t* kb = a.k_pages + ph * ps * D;
    uint8_t* vb = a.v_pages + ph * ps * D;
    if (held > 0) {
      if (k_scale > k_old)
        for (int i = tid; i < held * D / 8; i += threads)
          reinterpret_cast<uint2*>(kb)[i] = rescale_codes(reinterpret_cast<uint2*>(kb)[i], k_old / k_scale);
      if (v_scale > v_old)
        for (int i = tid; i < held * D / 8; i += threads)
          reinterpret_cast<uint2*>(vb)[i] = rescale_codes(reinterpret_cast<uint2*>(vb)[i], v_old / v_scale);
    }
    if (on) {
      store_codes(kb + slot * D, u, xk, 1.f / k_scale);
      float xv[16];
      unpack(wv, xv);
      store_codes(vb + slot * D, u, xv, 1.f / v_scale);
    }
    if (tid == 0) {
      // every thread read the old scales before the barrier above
      a.k_scales[ph] = k_scale;
      a.v_scales[ph] = v_scale;
    }
  }
}

template <int D>
int launch_append_d(AppendArgs a, cudaStream_t stream) {
  const PagedBatchDev& b = a.batch;
  cudaError_t e;
  if (b.max_q == 1) {
    constexpr int kHeadsPerWarp = 512 / D;
    const long long warps = static_cast<long long>(b.B) * (a.Hkv + (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp);
    const long long blocks = (warps + 3) / 4;
    if (blocks > 0x7fffffffLL) return -1;
    e = launch_overlapped(append_one_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, a);
  } else {
    a.kv_parts = (a.Hkv + kHeadsPerBlock - 1) / kHeadsPerBlock;
    a.q_parts = (a.Hq + kQHeadsPerBlock - 1) / kQHeadsPerBlock;
    // Blocks per sequence for the longest one, or, where that would leave most
    // blocks of a ragged batch without work, as many items as the packed rows
    // can touch pages, each of which looks for its sequence.
    const long long slots = (static_cast<long long>(b.max_q) + b.page_size - 2) / b.page_size + 1;
    const long long packed = b.T / b.page_size + 2LL * b.B;
    long long items = slots * b.B;
    a.page_slots = static_cast<int>(slots);
    if (items > 2 * packed && b.cu_q != nullptr) {
      items = packed;
      a.page_slots = 0;
    }
    const long long blocks = items * (a.kv_parts + a.q_parts);
    if (blocks > 0x7fffffffLL) return -1;
    e = launch_overlapped(append_pages_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(b.page_size * (D / 16)), 0,
                          stream, a);
  }
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace

int launch_paged_append(const PagedPool& pool, const PagedBatchDev& batch, const PagedAppend& p,
                        cudaStream_t stream) {
  AppendArgs a{};
  a.batch = batch;
  a.k = static_cast<const __nv_bfloat16*>(p.k);
  a.v = static_cast<const __nv_bfloat16*>(p.v);
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.q_out = static_cast<__nv_bfloat16*>(p.q_out);
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.q_stride = p.q_stride;
  a.q_out_stride = p.q_out_stride;
  a.k_pages = static_cast<uint8_t*>(pool.k_pages);
  a.v_pages = static_cast<uint8_t*>(pool.v_pages);
  a.k_scales = pool.k_scales;
  a.v_scales = pool.v_scales;
  a.cos = p.cos;
  a.sin = p.sin;
  a.Hq = p.Hq;
  a.Hkv = pool.num_heads;
  a.rot = p.rot;
  a.max_pos = p.max_pos;
  a.interleaved = p.interleaved;
  a.status = device_status_word();
  if (!a.status) return -3;
  return pool.d == 64 ? launch_append_d<64>(a, stream) : launch_append_d<128>(a, stream);
}

}  // namespace fa
