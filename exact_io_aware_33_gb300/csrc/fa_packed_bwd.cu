// Gradients of attention over packed sequences with grouped heads.
//
// Mathematics, with the forward's O and LSE and the loss's gradient dO, per
// query row i (a token's head) and key j that it sees:
//   D_i = sum_c dO_ic O_ic,  P_ij = e^(scale q_i . k_j - LSE_i),
//   dS_ij = P_ij (dO_i . v_j - D_i),
//   dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij q_i  (over the group's heads too),
//   dQ_i = scale sum_j dS_ij k_j.
// P and dS are rounded to bf16 for the products (2^-9 of a term on average);
// everything else is fp32.
//
// A row that sees one key, its own (a window of 1, a sequence of one token), needs no
// tiles: it is computed as it is written, beside the row sums, with dO . v - D as sum_c
// dO_c (v_c - O_c). That is exactly 0 where O is v, as the forward leaves it, where two
// sums would leave their rounding errors.
//
// Three kernels: D; dK and dV, with a key tile resident and the tiles of query
// rows streamed; dQ, with a tile of query rows resident and the key tiles
// streamed. S and dP are computed in both, 7 products instead of the 5 of a
// single kernel, which would add its dQ tiles up in memory: with fp32 atomics,
// in an order that changes from run to run (a workspace of 4 T Hq d bytes, its
// clearing and its conversion with it). Here every sum has its owner and a
// fixed order, so the same inputs give the same bits.
//
// dK, dV: thread = key row = tensor-memory lane, S^T = K Q^T and dP^T = V dO^T
// with both operands in shared memory, P^T and dS^T left in tensor memory as the
// first operands of dV += P^T dO and dK += dS^T Q: no probability goes through
// shared memory. At d = 64 P and dS have columns of their own; one warp issues
// S^T and dP^T, each as soon as its predecessor is in registers, and another dV
// and dK, neither waiting for the other's order. At d = 128 there are no columns
// for that: P and dS lie over S and dP, and one warp issues dV, the next S^T, dK,
// the next dP^T: the exponentials are formed under dK and dP^T, dS under dV and
// S^T. dQ: thread = query row, S and dP leave for registers at once, dS has
// columns of its own, and two warps issue.
//
// Sixteen warps form P and dS (a quarter of a tile's columns per warpgroup), four
// write the accumulators back while the next item is at work, and a helper brings
// the row statistics. Tiles (fa_packed.cuh) hold a key head's whole group. What a
// box reaches past its sequence belongs to another one and may hold anything;
// where it would be multiplied by 0 the helper puts zeros in its place, in shared
// memory, before the tile is handed to the tensor core.
//
// What bounds it: 14 d flops per visible pair on the tensor core (10 d of them
// the algorithm's), which reads up to 128 bytes a clock of operands from shared
// memory, two exponentials per pair, and the hand-offs between the roles: a step
// of 128 x 128 takes 2730 (dK, dV) and 1940 (dQ) cycles at d = 128, 2230 and 1630
// at d = 64 (medians under time stamps, which cost some), of which the tensor core is at work for
// 2200, 1650, 1100 and 820.
// Measured (a CUDA graph of the call, replayed back to back; one call after another from
// Python the d = 128 ones take 5 to 7 % more, under the power limit): 8 documents of up to
// 4096 tokens, 32 / 8 heads, d = 128: 588 us, 1020 TFLOP/s of the algorithm's; one of 8192,
// 16 heads: 589, 1167; 24 images of up to 1369 tokens, 16 heads, d = 64, unmasked: 269, 625.
// dK and dV's work is divided by key tiles and key heads only. Where one key head serves
// many heads, the first keys' item is what the call takes: one sequence of 11585 tokens,
// 8 / 1 heads, 1178 us, 583 TFLOP/s; one of 8192, 32 / 1, 3184 us, 432 (d = 128, causal).

#include <algorithm>

#include "fa_packed.cuh"

namespace fa {
namespace {

// Steps and items counted are not negative; said so, their remainders and quotients
// take fewer instructions (269.5 us instead of 270.6, 24 images of up to 1369 tokens).
__device__ __forceinline__ uint32_t u32(int x) { return static_cast<uint32_t>(x); }

constexpr int kKT = kKeyTile;  // keys per tile; also rows per tile of query rows
constexpr int kItems = 4;      // item records kept
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 bf16, 128-byte swizzled
// Warps 0-15 compute (warpgroup w: columns [32 w, 32 w + 32) of S and dP), 16 and 17 issue MMAs, 18 loads, 19 helps,
// 20-23 write back.
constexpr int kComputeWarps = 16, kMmaWarp = 16, kSumWarp = 17, kLoadWarp = 18, kHelpWarp = 19, kOutWarp = 20;
constexpr int kThreads = 768;
constexpr int kCols = 32;
// Registers per thread, of the 80 that the CTA is launched with: 512 x 88 + 256 x 64 = 768 x 80.
constexpr int kComputeRegs = 88, kOtherRegs = 64;
constexpr float kLog2e = 1.4426950408889634f;

// An item, left by the TMA warp.
struct Item {
  int end;      // 1: no more items (the rest is not set)
  int row0, n;  // the sequence's first row, and its length
  int h;        // key head
  int x0;       // first token of the resident tile
  int t0, ns;   // first streamed tile, and how many
  int pad;
};

struct BwdArgs {
  PackedShape s;
  PackedList list;
  const float* neg_lse;  // [Hkv, T, G], log2 units
  const float* neg_d;    // [Hkv, T, G]
  __nv_bfloat16* out[2];   // dK, dV; or dQ
  long long out_stride[2];
  int* status;
  float scale, scale_log2;
};

template <int D, bool kKeys>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  // stages of the streamed pair, Q and dO (dK, dV) or K and V (dQ): what there is room for
  static constexpr int kStages0 = D == 64 ? 4 : kKeys ? 2 : 3, kStages1 = D == 64 ? 4 : 2;
  static constexpr int kStatStages = D == 64 ? 4 : 2;
  static constexpr int kResOff = 0;  // resident pairs of tiles: K and V, or Q and dO (d = 64: the next item's too)
  static constexpr int kResBufs = D == 64 ? 2 : 1;
  static constexpr int kRing0 = kResBufs * 2 * kTileBytes, kRing1 = kRing0 + kStages0 * kTileBytes;
  static constexpr int kStatOff = kRing1 + kStages1 * kTileBytes;  // dK, dV: per stage 128 -LSE, 128 -D
  static constexpr int kOutOff = kStatOff + (kKeys ? kStatStages * 1024 : 0);
  static constexpr bool kStaged = D == 64 || kKeys;  // write-back by way of 2 KiB per warp (dQ, d = 128: no room)
  static constexpr int kItemOff = kOutOff + (kStaged ? 4 * 2048 : 0);
  static constexpr int kBarOff = kItemOff + kItems * static_cast<int>(sizeof(Item));
  // P and dS have columns of their own, so that S and dP are computed by one
  // warp's issue and used by another's, neither waiting for the other's order.
  // (dK, dV at d = 128: no room; one warp issues all products in a fixed order.)
  static constexpr bool kApart = D == 64 || !kKeys;
  static constexpr int kIssuers = kApart ? 2 : 1;
  enum : int {
    kBarResFull = 0,
    kBarResFree = kBarResFull + kResBufs,
    kBarLoad0 = kBarResFree + kResBufs,   // a stage's tile has landed
    kBarEmpty0 = kBarLoad0 + kStages0,    // and is not needed any more
    kBarReady = kBarEmpty0 + kStages0,    // the helper is done with the step
    kBarLoad1 = kBarReady + kStages0,
    kBarEmpty1 = kBarLoad1 + kStages1,
    kBarS = kBarEmpty1 + kStages1,
    kBarDp,
    kBarP,       // dK, dV: P is written; dQ: S is in registers
    kBarDpFree,  // dQ: dP is in registers
    kBarDs,      // dS is written
    kBarDsFree,  // and has been read, and P of its step (where they are apart)
    kBarFinal,   // an item's accumulators are complete
    kBarAccFree, // and have been read out
    kBarItemFull,
    kBarItemEmpty = kBarItemFull + kItems,
    kBarDrain = kBarItemEmpty + kItems,  // two
    kNumBars = kBarDrain + 2
  };
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16;
  // Tensor-memory columns: S, dP, then dK and dV, or dQ; P and dS, 64 each, where they are apart.
  enum : uint32_t { kColS = 0, kColDp = 128, kColA = 256, kColP = 384, kColDs = 448 };
  static_assert(kSmemBytes <= 232448, "tiles exceed shared memory");
  static_assert(kItemOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

// ---------------------------------------------------------------- D
// -D = -rowsum(dO O) and -LSE in log2 units for every row and head, read as they
// lie and laid out so that the rows of a tile are contiguous; d / 8 lanes per row.
// Bound by memory: 4 d + 12 bytes a row (37 us for 12400 tokens of 32 heads, d =
// 128, 207 MB). Many threads with two rows each keep more loads in flight than fewer
// with four or eight (the call: 588 us, 605 and 662). The first blocks make the lists of
// the two kernels that follow, and the next ones compute the rows of own_rows, under the
// others' loads.
constexpr int kSumThreads = 512;

struct SumArgs {
  PackedShape s;
  PackedList lists[2];
  int n_lists;
  int n_own;  // blocks of own_rows
  int* status;
  // for own_rows
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *dq, *dk, *dv;
  long long q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride;
  float scale, scale_log2;
};

// N channels of a lane: N / 2 words, in fp32 and back.
template <int N>
struct Channels {
  float x[N];
  __device__ __forceinline__ explicit Channels(float f) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = f;
  }
  __device__ __forceinline__ Channels(const __nv_bfloat16* at, int lane) {
    uint32_t w[N / 2];
    if constexpr (N == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(at + lane * N);
      w[0] = u.x;
      w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(at + lane * N);
    }
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
      x[2 * c] = __uint_as_float(w[c] << 16);
      x[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* at, int lane, float f) const {
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(at + lane * N) = make_uint2(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f));
    else
      *reinterpret_cast<uint32_t*>(at + lane * N) = pack_bf16(x[0] * f, x[1] * f);
  }
  __device__ __forceinline__ void add(float f, const Channels& y) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = fmaf(f, y.x[c], x[c]);
  }
};

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// The gradients of the rows that see their own key alone: all tokens where the
// window is 1, otherwise the sequences of one token. A warp takes a key head of up
// to kOwn of them, its lanes the channels. Bound by the latency of a warp's chain of
// loads and sums, a head at a time: 4096 sequences of one token, 12 / 4 heads, d = 64,
// 24.6 us for the call (6 x up to 5001 tokens with a window of 1: 68 us for 204 MB).
// Found out by the row sums' own threads instead, which rows these are cost 10 us of
// 590 and 10 of 269 in calls that have none, and by the tile kernels 8 of 269.
constexpr int kOwn = 8;
constexpr int kSumWarps = kSumThreads / 32;

// Warps' items: below 2^31, as T Hq and B Hkv are.
__host__ __device__ __forceinline__ int own_items(const PackedShape& s, int count) { return (count + kOwn - 1) / kOwn * s.Hkv; }

template <int D>
__device__ __forceinline__ void own_rows(const SumArgs& a, const __nv_bfloat16* o, const __nv_bfloat16* dO,
                                         long long do_stride, const float* lse, int block) {
  using Part = Channels<D / 32>;
  const PackedShape& s = a.s;
  const int lane = static_cast<int>(lane_id()), G = s.by_group.G;
  int first = 0, count = s.B;
  if (s.window == 1) {
    for (int b = block * kSumThreads + static_cast<int>(threadIdx.x); b < s.B; b += a.n_own * kSumThreads)
      packed_seq<true>(s, b, a.status);  // (reports borders that are wrong)
    first = min(max(s.cu[0], 0), s.T);
    count = max(min(s.cu[s.B], s.T) - first, 0);
  }
  const int items = own_items(s, count);
#pragma unroll 1
  for (int i = block * kSumWarps + warp_id(); i < items; i += a.n_own * kSumWarps) {
    const int set = s.by_head.div(i), h = i - set * s.Hkv, mine = set * kOwn + lane;
    int token = -1;
    if (lane < kOwn && mine < count) {
      if (s.window == 1) {
        token = first + mine;
      } else {
        const PackedSeq q = packed_seq<true>(s, mine, a.status);
        if (q.n == 1) token = q.row0;
      }
    }
#pragma unroll 1
    for (uint32_t left = __ballot_sync(0xffffffffu, token >= 0); left; left &= left - 1) {
      const long long t = __shfl_sync(0xffffffffu, token, __ffs(left) - 1);
      const Part k(a.k + t * a.k_stride + static_cast<long long>(h) * D, lane);
      const Part v(a.v + t * a.v_stride + static_cast<long long>(h) * D, lane);
      Part dk(0.f), dv(0.f);
#pragma unroll 1
      for (int g = 0; g < G; ++g) {
        const long long head = static_cast<long long>(h) * G + g, row = t * s.Hq + head;
        const Part q(a.q + t * a.q_stride + head * D, lane), out(o + row * D, lane), grad(dO + t * do_stride + head * D, lane);
        float score = 0.f, diff = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          score = fmaf(q.x[c], k.x[c], score);
          diff = fmaf(grad.x[c], v.x[c] - out.x[c], diff);
        }
        const float p = ex2(fmaf(warp_total(score), a.scale_log2, -kLog2e * lse[row]));
        const float ds = p * warp_total(diff);
        k.store(a.dq + t * a.dq_stride + head * D, lane, ds * a.scale);
        dk.add(ds, q);
        dv.add(p, grad);
      }
      dk.store(a.dk + t * a.dk_stride + static_cast<long long>(h) * D, lane, a.scale);
      dv.store(a.dv + t * a.dv_stride + static_cast<long long>(h) * D, lane, 1.f);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kSumThreads, 4) packed_rowsum_kernel(const __nv_bfloat16* __restrict__ o,
                                                                    const __nv_bfloat16* __restrict__ dO,
                                                                    long long do_stride, const float* __restrict__ lse,
                                                                    float* __restrict__ neg_lse, float* __restrict__ neg_d,
                                                                    GroupDiv by_token, long long rows,
                                                                    const __grid_constant__ SumArgs args) {
  constexpr int kLanes = D / 8, kUnroll = 2;
  grid_dep_wait();
  grid_dep_launch();
  if (static_cast<int>(blockIdx.x) < args.n_lists) {
    make_list<kSumThreads>(args.s, args.lists[blockIdx.x], args.status);
    return;
  }
  const int block = static_cast<int>(blockIdx.x) - args.n_lists - args.n_own;
  if (block < 0) {
    own_rows<D>(args, o, dO, do_stride, lse, block + args.n_own);
    return;
  }
  const GroupDiv group = args.s.by_group;
  const int Hq = args.s.Hq;
  const int lane = threadIdx.x % kLanes;
  const long long per = kSumThreads / kLanes, first = block * per * kUnroll + threadIdx.x / kLanes;
  uint4 a[kUnroll], b[kUnroll];
  float l[kUnroll];
  long long to[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long row = first + i * per;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    l[i] = 0.f;
    if (row < rows) {
      const int t = by_token.div(static_cast<int>(row)), hq = static_cast<int>(row) - t * Hq;
      a[i] = *reinterpret_cast<const uint4*>(o + row * D + lane * 8);
      b[i] = *reinterpret_cast<const uint4*>(dO + t * do_stride + static_cast<long long>(hq) * D + lane * 8);
      l[i] = lse[row];
      const int h = group.div(hq);
      to[i] = (static_cast<long long>(h) * args.s.T + t) * group.G + (hq - h * group.G);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, y[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
      sum = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), sum);
    }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const long long row = first + i * per;
    if (lane == 0 && row < rows) {
      neg_d[to[i]] = -sum;
      neg_lse[to[i]] = -kLog2e * l[i];
    }
  }
}

// ---------------------------------------------------------------- shared parts
// Bits c of a word for lo <= c < hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : (1u << max(hi, 0)) - 1u;
  const uint32_t skip = lo >= 32 ? 0xffffffffu : (1u << max(lo, 0)) - 1u;
  return below & ~skip;
}

// 32 fp32 accumulator columns of this thread's row to bf16, in 16-byte units.
__device__ __forceinline__ uint4 unit_of(const uint32_t (&x)[32], float f, int v) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = pack_bf16(__uint_as_float(x[8 * v + 2 * e]) * f, __uint_as_float(x[8 * v + 2 * e + 1]) * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Writes them for a warp's 32 rows, by way of its staging block: 64-byte rows,
// whose 16-byte units change places with the row, so that neither side meets a
// bank twice. Four lanes then write a row's 64 bytes. row_at(r): where the
// columns of row r go, or null.
template <typename RowAt>
__device__ __forceinline__ void store_staged(const uint32_t (&x)[32], float f, uint8_t* stage, int lane, RowAt row_at) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) * 16)) = unit_of(x, f, v);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 8 * j + (lane >> 2), v = lane & 3;
    const uint4 val = *reinterpret_cast<const uint4*>(stage + r * 64 + ((v ^ ((r >> 1) & 3)) * 16));
    __nv_bfloat16* to = row_at(r);
    if (to != nullptr) *reinterpret_cast<uint4*>(to + v * 8) = val;
  }
  __syncwarp();  // the block is read back before it is written again
}

// Writes them straight to this thread's row, or nowhere.
__device__ __forceinline__ void store_direct(const uint32_t (&x)[32], float f, __nv_bfloat16* to) {
  if (to == nullptr) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(to + 8 * v) = unit_of(x, f, v);
}

// Makes x[c] zero where bit c of `keep` is not set.
__device__ __forceinline__ void keep_bits(float2* x, uint32_t keep) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    if (!((keep >> (2 * c)) & 1u)) x[c].x = 0.f;
    if (!((keep >> (2 * c + 1)) & 1u)) x[c].y = 0.f;
  }
}

__device__ __forceinline__ float2 pair(const uint32_t* x) { return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])); }

// The CTA's barriers and tensor memory, the item records, and the TMA warp's
// loop, which the two kernels share: kKeys: K and V resident, Q and dO streamed.
template <int D, bool kKeys>
struct Frame {
  using C = Cfg<D, kKeys>;
  uint8_t* smem;
  uint32_t base, tmem;
  volatile int* abort_flag;
  volatile int* loaded;  // stream steps that the TMA warp has started

  __device__ __forceinline__ uint32_t bar(int i) const { return base + C::kBarOff + 8u * i; }
  __device__ __forceinline__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(smem + C::kMiscOff); }
  __device__ __forceinline__ Item* items() const { return reinterpret_cast<Item*>(smem + C::kItemOff); }
  __device__ __forceinline__ uint8_t* ring0(int g) const { return smem + C::kRing0 + u32(g) % C::kStages0 * C::kTileBytes; }
  __device__ __forceinline__ uint8_t* ring1(int g) const { return smem + C::kRing1 + u32(g) % C::kStages1 * C::kTileBytes; }
  // Waits of stream step g on the barriers of its stages.
  __device__ __forceinline__ bool landed0(int g) const { return at_step(C::kBarLoad0, C::kStages0, g); }
  __device__ __forceinline__ bool landed1(int g) const { return at_step(C::kBarLoad1, C::kStages1, g); }
  __device__ __forceinline__ bool ready(int g) const { return at_step(C::kBarReady, C::kStages0, g); }
  __device__ __forceinline__ bool at_step(int b, int stages, int g) const {
    return mbar_wait_w(bar(b + u32(g) % stages), (u32(g) / stages) & 1, abort_flag);
  }
  // The same for the compute warps. At d = 128 they wait for the tensor core most
  // of the time, and asleep they take no issue slots and shared-memory cycles from
  // it (588 us instead of 599, 8 documents of up to 4096 tokens, 32 / 8 heads); at d =
  // 64 they are what is waited for (269 instead of 280, 24 images of up to 1369).
  __device__ __forceinline__ bool wait_calm(int b, int g) const {
    return D == 64 ? mbar_wait_w(bar(b), g & 1, abort_flag) : mbar_wait_sleep_w(bar(b), g & 1, abort_flag);
  }
  // Step g's statistics may be written: dK of the step that had their place before has gone.
  __device__ __forceinline__ bool stats_free(int g) const {
    return g < C::kStatStages || at_step(C::kBarEmpty0, C::kStages0, g - C::kStatStages);
  }
  __device__ __forceinline__ bool resident(int q) const { return at_step(C::kBarResFull, C::kResBufs, q); }
  // The g-th phase of a barrier that has one per step.
  __device__ __forceinline__ bool wait(int b, int g) const { return mbar_wait_w(bar(b), g & 1, abort_flag); }
  __device__ __forceinline__ float* stats(int g) const {
    return reinterpret_cast<float*>(smem + C::kStatOff + u32(g) % C::kStatStages * 1024);
  }

  // The dQ kernel does not read what the one before it on the stream writes, so it
  // does not wait for it here, but at its end (close): its CTAs take the SMs that
  // dK and dV's leave. What it does read is complete: that kernel's CTAs let it
  // start only after their own wait.
  __device__ __forceinline__ void open(uint8_t* raw, const PackedShape& s) {
    base = smem_u32(raw);  // 1 KiB aligned, as the array is declared (there is no room to align it here)
    smem = raw;
    abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    loaded = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 8);
    if (threadIdx.x == 0) {
      for (int i = C::kBarResFull; i < C::kBarLoad0; ++i) mbar_init(bar(i), 1);
      for (int i = C::kBarLoad0; i < C::kBarS; ++i)
        // (dK, dV's helper: each lane's copies, and what the warp wrote itself)
        mbar_init(bar(i), kKeys && i >= C::kBarReady && i < C::kBarLoad1 ? 33 : 1);
      mbar_init(bar(C::kBarS), kKeys ? 2 : 1);  // dK, dV: and the MMA warp, which passes on that the statistics are written
      mbar_init(bar(C::kBarDp), 1);
      mbar_init(bar(C::kBarP), kComputeWarps);
      mbar_init(bar(C::kBarDpFree), kComputeWarps);
      mbar_init(bar(C::kBarDs), kComputeWarps);
      mbar_init(bar(C::kBarDsFree), 1);
      mbar_init(bar(C::kBarFinal), 1);
      mbar_init(bar(C::kBarAccFree), 4);
      for (int i = 0; i < kItems; ++i) {
        mbar_init(bar(C::kBarItemFull + i), 1);
        mbar_init(bar(C::kBarItemEmpty + i), kComputeWarps + C::kIssuers + 5);  // and the helper and write-back warps
      }
      mbar_init(bar(C::kBarDrain), 1);
      mbar_init(bar(C::kBarDrain + 1), 1);
      *abort_flag = 0;
      *loaded = 0;
      mbar_fence_init();
    }
    if (warp_id() == kMmaWarp) {
      tmem_alloc(smem_u32(tmem_slot()), 512);
      tmem_relinquish();
    }
    if (kKeys && s.tpt * s.by_group.G < 128) {
      // rows that no box of query rows reaches: summed over as the others are
      for (int i = 0; i < C::kStages0 + C::kStages1; ++i)
        zero_rows(smem + C::kRing0 + i * C::kTileBytes, kChunkBytes, C::kChunks, s.tpt * s.by_group.G, 128,
                  threadIdx.x, kThreads);
      fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *tmem_slot();
    if (kKeys) {
      grid_dep_wait();
      grid_dep_launch();
    }
  }

  // Item number k, for a consuming warp that gives it back with give_item.
  __device__ __forceinline__ bool get_item(int k) const {
    return mbar_wait_w(bar(C::kBarItemFull + u32(k) % kItems), (u32(k) / kItems) & 1, abort_flag);
  }
  __device__ __forceinline__ void give_item(int k) const { mbar_arrive_warp(bar(C::kBarItemEmpty + u32(k) % kItems)); }

  // Whether stream step t0 + jj of an item is a tile that reaches past the sequence.
  __device__ __forceinline__ static bool last_tile(const PackedShape& s, const Item& it, int jj) {
    return (it.t0 + jj + 1) * (kKeys ? s.tpt : kKT) > it.n;
  }

  // The TMA warp; counts the loads of the resident tiles and of stages that it started.
  __device__ __forceinline__ void produce(const PackedShape& s, const PackedList& list, const CUtensorMap* res0,
                                          const CUtensorMap* res1, const CUtensorMap* str0, const CUtensorMap* str1,
                                          int* status, int* res_loads, int (&stage_loads)[2]) {
    ItemQueue queue;
    queue.start(s, list, status);
    if (lane_id() != 0) return;
    tma_prefetch_map(res0);
    tma_prefetch_map(res1);
    tma_prefetch_map(str0);
    tma_prefetch_map(str1);
    const uint32_t rows_bytes = static_cast<uint32_t>(s.tpt * s.by_group.G * 128 * C::kChunks);
    const uint32_t res_bytes = 2 * (kKeys ? C::kTileBytes : rows_bytes), str_bytes = kKeys ? rows_bytes : C::kTileBytes;
    bool ok = true;
    int g = 0, q = 0;
    PackedEntry e;
    int h;
    while (ok && queue.take(&e, &h)) {
      const int x1 = min(e.i0 + list.unit, e.n);
      const TileRange r = kKeys ? rows_of(s, e.n, e.i0, x1) : keys_of(s, e.n, e.i0, x1);
      const Item it{0, e.row0, e.n, h, e.i0, r.lo, r.n, 0};
      if (q >= kItems) ok = mbar_wait(bar(C::kBarItemEmpty + u32(q) % kItems), (u32(q) / kItems - 1) & 1, abort_flag);
      if (!ok) break;
      items()[u32(q) % kItems] = it;
      mbar_arrive(bar(C::kBarItemFull + u32(q) % kItems));
      auto load_resident = [&]() {
        const int rb = u32(q) % C::kResBufs;
        if (q >= C::kResBufs) ok = mbar_wait(bar(C::kBarResFree + rb), (u32(q) / C::kResBufs - 1) & 1, abort_flag);
        if (!ok) return;
        const uint32_t res = base + C::kResOff + rb * 2 * C::kTileBytes, res_full = bar(C::kBarResFull + rb);
        mbar_arrive_expect_tx(res_full, res_bytes);
        for (int c = 0; c < C::kChunks; ++c) {
          tma_load_4d(res + c * kChunkBytes, res0, res_full, c * 64, 0, h, e.row0 + e.i0);
          tma_load_4d(res + C::kTileBytes + c * kChunkBytes, res1, res_full, c * 64, 0, h, e.row0 + e.i0);
        }
        *res_loads = q + 1;
      };
      // a second buffer is free before the ring's next stage is, the only one after it
      if (C::kResBufs > 1) load_resident();
      for (int jj = 0; jj < it.ns && ok; ++jj, ++g) {
        const int row = e.row0 + (it.t0 + jj) * (kKeys ? s.tpt : kKT);
        queue.step(it.ns - jj);
        auto load = [&](int w, int load_bar, int empty_bar, int stages, uint8_t* to) {
          if (g >= stages) ok = mbar_wait(bar(empty_bar + u32(g) % stages), (u32(g) / stages - 1) & 1, abort_flag);
#ifdef FA_TEST_SKIP_ARRIVE
          // Test-only build (never in libfa.so): the first item's last tile (Q, or
          // K) is never loaded and nothing more is, so the bounded waits for it
          // run out and the CTA winds down through the abort path.
          if (w == 0 && jj == it.ns - 1) ok = false;
#endif
          if (!ok) return;
          const uint32_t full = bar(load_bar + u32(g) % stages);
          mbar_arrive_expect_tx(full, str_bytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(smem_u32(to) + c * kChunkBytes, w == 0 ? str0 : str1, full, c * 64, 0, h, row);
          stage_loads[w] = g + 1;
        };
        load(1, C::kBarLoad1, C::kBarEmpty1, C::kStages1, ring1(g));
        if (ok) load(0, C::kBarLoad0, C::kBarEmpty0, C::kStages0, ring0(g));
        *loaded = g + 1;
        if (C::kResBufs == 1 && jj == 0 && ok) load_resident();
      }
      ++q;
    }
    if (ok && q >= kItems) ok = mbar_wait(bar(C::kBarItemEmpty + u32(q) % kItems), (u32(q) / kItems - 1) & 1, abort_flag);
    if (ok) {
      items()[u32(q) % kItems].end = 1;
      mbar_arrive(bar(C::kBarItemFull + u32(q) % kItems));
    }
  }

  // The write-back warps: per item, body(item, put) calls put(which, factor,
  // row_at) for each accumulator; row_at(r): where row r of this warp's 32 goes,
  // or null. They have the accumulators' columns read out while the compute warps
  // are at the next item's first P, which the next products into them wait for.
  template <typename Body>
  __device__ __forceinline__ void write_back(Body body) const {
    constexpr int kAcc = kKeys ? 2 : 1;
    const int warp = warp_id(), lane = lane_id();
    const uint32_t acc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kColA;
    [[maybe_unused]] uint8_t* stage = smem + C::kOutOff + (warp & 3) * 2048;
    for (int q = 0;; ++q) {
      if (!get_item(q) || items()[u32(q) % kItems].end) break;
      const Item it = items()[u32(q) % kItems];
      give_item(q);
      // (a whole item: with a token of 128 heads a step, a million tokens are more than a second)
      if (!mbar_wait_long_w(bar(C::kBarFinal), q & 1, abort_flag, loaded)) break;
      tc_fence_after();
      body(it, [&](int which, float factor, auto&& row_at) {
        [[maybe_unused]] __nv_bfloat16* mine = C::kStaged ? nullptr : row_at(lane);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          tmem_ld32(acc + which * D + c, x);
          tmem_ld_wait(x);
          if (which == kAcc - 1 && c == D - 32) {
            tc_fence_before();
            mbar_arrive_warp(bar(C::kBarAccFree));
          }
          if constexpr (C::kStaged)
            store_staged(x, factor, stage, lane, [&](int r) { __nv_bfloat16* to = row_at(r); return to != nullptr ? to + c : to; });
          else
            store_direct(x, factor, mine != nullptr ? mine + c : nullptr);
        }
      });
    }
  }

  // Lets every MMA that an issuing warp issued finish, before TMEM is released.
  __device__ __forceinline__ void drain(int which) const {
    mma_commit_w(bar(C::kBarDrain + which));
    mbar_wait_w(bar(C::kBarDrain + which), 0, nullptr);
  }

  __device__ __forceinline__ void close(int res_loads, const int (&stage_loads)[2], int* status) {
    tc_fence_before();
    __syncthreads();
    if (warp_id() == kLoadWarp && lane_id() == 0 && *abort_flag) {
      // Every role has stopped, so the flag is final: let every copy this
      // thread started land before the CTA exits (only the last load of each
      // buffer can still be pending).
      for (int i = max(res_loads - C::kResBufs, 0); i < res_loads; ++i)
        mbar_wait(bar(C::kBarResFull + u32(i) % C::kResBufs), (u32(i) / C::kResBufs) & 1, nullptr);
      for (int i = max(stage_loads[0] - C::kStages0, 0); i < stage_loads[0]; ++i)
        mbar_wait(bar(C::kBarLoad0 + u32(i) % C::kStages0), (u32(i) / C::kStages0) & 1, nullptr);
      for (int i = max(stage_loads[1] - C::kStages1, 0); i < stage_loads[1]; ++i)
        mbar_wait(bar(C::kBarLoad1 + u32(i) % C::kStages1), (u32(i) / C::kStages1) & 1, nullptr);
    }
    if (warp_id() == kMmaWarp) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(status, kStatusTimeout);
    if (!kKeys) {  // (so that whoever waits for this kernel has waited for dK and dV's as well)
      grid_dep_launch();
      grid_dep_wait();
    }
  }
};

// ---------------------------------------------------------------- dK, dV
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkv_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                      const __grid_constant__ BwdArgs args) {
  using F = Frame<D, true>;
  using C = typename F::C;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const PackedShape& sh = args.s;
  const int G = sh.by_group.G;
  F f;
  f.open(smem_raw, sh);
  const int warp = warp_id(), lane = lane_id();
  if (warp >= kComputeWarps) regs_decrease<kOtherRegs>();
  int res_loads = 0, stage_loads[2] = {0, 0};

  if (warp == kLoadWarp) {
    f.produce(sh, args.list, &tmK, &tmV, &tmQ, &tmDo, args.status, &res_loads, stage_loads);
  } else if (warp == kHelpWarp) {
    // ------------------------------------------------------------ statistics
    // Each step's 128 -LSE and -D are copied without being waited for: they arrive
    // on the stage's barrier themselves (588 us instead of 592, 8 documents of up to
    // 4096 tokens; as much as a load from memory takes each step, where L2 does not
    // hold them). Rows that are none get zeros: their queries and dO are zeros too, so P = 1 adds nothing.
    bool ok = true;
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const Item it = f.items()[u32(q) % kItems];
      f.give_item(q);
      for (int jj = 0; jj < it.ns; ++jj, ++g) {
        const int i0 = (it.t0 + jj) * sh.tpt, rows = min(sh.tpt, it.n - i0) * G;
        const long long first = (static_cast<long long>(it.h) * sh.T + it.row0 + i0) * G;
        ok = f.stats_free(g);
        if (!ok) break;
        const uint32_t stat = smem_u32(f.stats(g));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          const long long at = first + min(r, rows - 1);
          cp_async_f32(stat + 4 * r, args.neg_lse + at, r < rows);
          cp_async_f32(stat + 512 + 4 * r, args.neg_d + at, r < rows);
        }
        if (F::last_tile(sh, it, jj)) {
          ok = f.landed0(g) && f.landed1(g);
          if (!ok) break;
          zero_rows(f.ring0(g), kChunkBytes, C::kChunks, rows, 128, lane, 32);
          zero_rows(f.ring1(g), kChunkBytes, C::kChunks, rows, 128, lane, 32);
          fence_async_smem();
        }
        // The copies arrive when they land, and that orders nothing else the lanes
        // wrote: the zeros are handed over by an arrival of their own, a release.
        cp_async_arrive(f.bar(C::kBarReady + u32(g) % C::kStages0));
        mbar_arrive_warp(f.bar(C::kBarReady + u32(g) % C::kStages0));
      }
    }
    cp_async_wait_all();
  } else if (warp == kMmaWarp || (C::kApart && warp == kSumWarp)) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdS = idesc_bf16_f32(kKT, 128, false, false);
    constexpr uint32_t kIdA = idesc_bf16_f32(kKT, D, false, true);
    constexpr uint64_t kTile = C::kTileBytes >> 4;
    const uint64_t res = sdesc_sw128(f.base + C::kResOff, 16, 1024);
    const uint64_t rows0 = sdesc_sw128(f.base + C::kRing0, 16, 1024), rows1 = sdesc_sw128(f.base + C::kRing1, 16, 1024);
    const uint64_t cols0 = sdesc_sw128(f.base + C::kRing0, kChunkBytes, 1024),
                   cols1 = sdesc_sw128(f.base + C::kRing1, kChunkBytes, 1024);
    const uint32_t tmem = f.tmem;
    bool ok = true;
    // S^T = K Q^T (which = 0) or dP^T = V dO^T (1) for stream step g, of item q
    auto issue_s = [&](int which, int q, int g) {
      const uint64_t a = res + (2 * (u32(q) % C::kResBufs) + which) * kTile;
      const uint64_t b = which ? rows1 + u32(g) % C::kStages1 * kTile : rows0 + u32(g) % C::kStages0 * kTile;
      mma_ss_depth_w<D>(tmem + (which ? C::kColDp : C::kColS), a, b, kIdS, 0u);
      mma_commit_w(f.bar(which ? C::kBarDp : C::kBarS));
      if (which == 0) mbar_arrive_warp(f.bar(C::kBarS));
    };
    // dV (+)= P^T dO (which = 1) or dK (+)= dS^T Q (0); where P and dS are not
    // apart, each warpgroup's part of them begins where its part of S or dP did
    auto issue_a = [&](int which, int g, bool first) {
      const uint64_t b = which ? cols1 + u32(g) % C::kStages1 * kTile : cols0 + u32(g) % C::kStages0 * kTile;
      const uint32_t col = C::kApart ? (which ? C::kColP : C::kColDs) : which ? C::kColS : C::kColDp;
      mma_ts_depth_w<!C::kApart>(tmem + C::kColA + which * D, tmem + col, b, kIdA, first ? 0u : 1u);
    };
    auto ready0 = [&](int g) { return f.landed0(g) && f.ready(g); };
    auto ready1 = [&](int g) { return f.landed1(g) && f.ready(g); };
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const int ns = f.items()[u32(q) % kItems].ns;
      f.give_item(q);
      if constexpr (C::kApart) {
        if (warp == kMmaWarp) {
          // S^T once its predecessor has become P, dP^T once its has become dS:
          // they are not needed before the compute warps are through with the other
          ok = f.resident(q);
          for (int jj = 0; jj < ns && ok; ++jj) {
            const int gs = g + jj;
            ok = (gs == 0 || f.wait(C::kBarP, gs - 1)) && ready0(gs);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, q, gs);
            ok = (gs == 0 || f.wait(C::kBarDpFree, gs - 1)) && ready1(gs);
            if (!ok) break;
            tc_fence_after();
            issue_s(1, q, gs);
          }
          if (ok) mma_commit_w(f.bar(C::kBarResFree + u32(q) % C::kResBufs));
        } else {
          // dV and dK; that dS is there says that S^T and dP^T have been computed
          for (int jj = 0; jj < ns && ok; ++jj) {
            const int gs = g + jj;
            ok = ready0(gs) && f.landed1(gs) && (jj > 0 || q == 0 || f.wait(C::kBarAccFree, q - 1)) && f.wait(C::kBarDs, gs);
            if (!ok) break;
            tc_fence_after();
            issue_a(1, gs, jj == 0);
            issue_a(0, gs, jj == 0);
            mma_commit_w(f.bar(C::kBarDsFree));
            mma_commit_w(f.bar(C::kBarEmpty0 + u32(gs) % C::kStages0));
            mma_commit_w(f.bar(C::kBarEmpty1 + u32(gs) % C::kStages1));
          }
          if (ok) mma_commit_w(f.bar(C::kBarFinal));
        }
      } else {
        ok = f.resident(q) && ready0(g);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, q, g);
        ok = f.landed1(g);
        if (!ok) break;
        tc_fence_after();
        issue_s(1, q, g);
        if (ns == 1) mma_commit_w(f.bar(C::kBarResFree + u32(q) % C::kResBufs));
        for (int jj = 0; jj < ns; ++jj) {
          const int gs = g + jj;
          ok = (jj > 0 || q == 0 || f.wait(C::kBarAccFree, q - 1)) && f.wait(C::kBarP, gs);
          if (!ok) break;
          tc_fence_after();
          issue_a(1, gs, jj == 0);
          mma_commit_w(f.bar(C::kBarEmpty1 + u32(gs) % C::kStages1));
          if (jj + 1 < ns) {
            ok = ready0(gs + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, q, gs + 1);
          }
          ok = f.wait(C::kBarDs, gs);
          if (!ok) break;
          tc_fence_after();
          issue_a(0, gs, jj == 0);
          mma_commit_w(f.bar(C::kBarEmpty0 + u32(gs) % C::kStages0));
          if (jj + 1 < ns) {
            ok = f.landed1(gs + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(1, q, gs + 1);
            // K and V are free once the item's last S^T and dP^T have completed
            if (jj + 2 == ns) mma_commit_w(f.bar(C::kBarResFree + u32(q) % C::kResBufs));
          } else {
            mma_commit_w(f.bar(C::kBarFinal));
          }
        }
      }
      g += ns;
    }
    f.drain(warp == kMmaWarp ? 0 : 1);
  } else if (warp >= kOutWarp) {
    // ------------------------------------------------------------ write-back
    f.write_back([&](const Item& it, auto&& put) {
      const int row = (warp & 3) * 32, n = it.n - it.x0 - row;  // this warp's first key, and keys from there on
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const long long stride = args.out_stride[which];
        __nv_bfloat16* out = args.out[which] + static_cast<long long>(it.row0 + it.x0 + row) * stride + static_cast<long long>(it.h) * D;
        put(which, which == 0 ? args.scale : 1.f, [&](int r) { return r < n ? out + r * stride : nullptr; });
      }
    });
  } else if (warp < kComputeWarps) {
    // ------------------------------------------------------------ P and dS
    regs_increase<kComputeRegs>();
    const int wg = warp / 4, row = threadIdx.x & 127;  // the group's queries are kCols wg .. kCols (wg + 1) - 1
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = f.tmem + lane_base + C::kColS + wg * kCols;
    const uint32_t tDp = f.tmem + lane_base + C::kColDp + wg * kCols;
    const uint32_t tP = C::kApart ? f.tmem + lane_base + C::kColP + wg * kCols / 2 : tS;
    const uint32_t tDs = C::kApart ? f.tmem + lane_base + C::kColDs + wg * kCols / 2 : tDp;
    const float2 sl2 = make_float2(args.scale_log2, args.scale_log2);
    bool ok = true;
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const Item& it = f.items()[u32(q) % kItems];  // (given back at the item's end)
      int i0 = it.t0 * sh.tpt;
      const int end = g + it.ns;
      // queries of a key k: [k, k + window); a border cuts the warp's part of a tile
      // that begins before token cut_lo, or from cut_hi on
      const int warp_k0 = it.x0 + (warp & 3) * 32;
      const int cut_lo = sh.causal ? warp_k0 + 31 - sh.by_group.div(wg * kCols) : -0x7fffffff;
      const int cut_hi = sh.window > 0 ? warp_k0 + sh.window - sh.by_group.div(wg * kCols + kCols - 1) : 0x7fffffff;
      for (; g < end; ++g, i0 += sh.tpt) {
        const float* stat = f.stats(g) + wg * kCols;
        const bool cut = i0 < cut_lo || i0 >= cut_hi;
        uint32_t seen = 0xffffffffu;
        if (cut) {
          const int k = it.x0 + row - i0;
          const int lo = sh.causal ? min(max(k, 0), 128) * G - wg * kCols : 0;
          const int hi = sh.window > 0 ? min(max(k + sh.window, 0), 128) * G - wg * kCols : kCols;
          seen = bits_between(lo, hi);
        }
        ok = f.wait_calm(C::kBarS, g);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[32], pk[16];
        float2 p[16];
        tmem_ld32(tS, x);
        tmem_ld_wait(x);
        if constexpr (C::kApart) {
          tc_fence_before();
          mbar_arrive_warp(f.bar(C::kBarP));
        }
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 l = *reinterpret_cast<const float4*>(stat + c);
          const float2 a = __ffma2_rn(pair(x + c), sl2, make_float2(l.x, l.y));
          const float2 b = __ffma2_rn(pair(x + c + 2), sl2, make_float2(l.z, l.w));
          p[c / 2] = make_float2(ex2(a.x), ex2(a.y));
          p[c / 2 + 1] = make_float2(ex2(b.x), ex2(b.y));
        }
        if (cut) keep_bits(p, seen);
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(p[c].x, p[c].y);
        if constexpr (C::kApart) {
          if (g > 0) ok = f.wait_calm(C::kBarDsFree, g - 1);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st16(tP, pk);
        if constexpr (!C::kApart) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(f.bar(C::kBarP));
        }
        ok = f.wait_calm(C::kBarDp, g);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tDp, x);
        tmem_ld_wait(x);
        if constexpr (C::kApart) {
          tc_fence_before();
          mbar_arrive_warp(f.bar(C::kBarDpFree));
        }
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 d = *reinterpret_cast<const float4*>(stat + 128 + c);
          p[c / 2] = __fmul2_rn(p[c / 2], __fadd2_rn(pair(x + c), make_float2(d.x, d.y)));
          p[c / 2 + 1] = __fmul2_rn(p[c / 2 + 1], __fadd2_rn(pair(x + c + 2), make_float2(d.z, d.w)));
        }
        if (cut) keep_bits(p, seen);  // (where a query is not seen, dP may be anything)
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(p[c].x, p[c].y);
        tmem_st16(tDs, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(f.bar(C::kBarDs));
      }
      if (!ok) break;
      f.give_item(q);
    }
  }
  f.close(res_loads, stage_loads, args.status);
}

// ---------------------------------------------------------------- dQ
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ BwdArgs args) {
  using F = Frame<D, false>;
  using C = typename F::C;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const PackedShape& sh = args.s;
  const int G = sh.by_group.G;
  F f;
  f.open(smem_raw, sh);
  const int warp = warp_id(), lane = lane_id();
  if (warp >= kComputeWarps) regs_decrease<kOtherRegs>();
  int res_loads = 0, stage_loads[2] = {0, 0};

  if (warp == kLoadWarp) {
    f.produce(sh, args.list, &tmQ, &tmDo, &tmK, &tmV, args.status, &res_loads, stage_loads);
  } else if (warp == kHelpWarp) {
    // ------------------------------------------------------------ keys past a sequence
    // (it takes part in every step: a warp that looked at some phases only could miss one)
    bool ok = true;
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const Item it = f.items()[u32(q) % kItems];
      f.give_item(q);
      for (int jj = 0; jj < it.ns; ++jj, ++g) {
        ok = f.landed0(g);
        if (!ok) break;
        if (F::last_tile(sh, it, jj)) {
          zero_rows(f.ring0(g), kChunkBytes, C::kChunks, it.n - (it.t0 + jj) * kKT, kKT, lane, 32);
          fence_async_smem();
        }
        mbar_arrive_warp(f.bar(C::kBarReady + u32(g) % C::kStages0));
      }
    }
  } else if (warp == kMmaWarp || warp == kSumWarp) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kKT, false, false);
    constexpr uint32_t kIdA = idesc_bf16_f32(128, D, false, true);
    constexpr uint64_t kTile = C::kTileBytes >> 4;
    const uint64_t res = sdesc_sw128(f.base + C::kResOff, 16, 1024);
    const uint64_t rows0 = sdesc_sw128(f.base + C::kRing0, 16, 1024), rows1 = sdesc_sw128(f.base + C::kRing1, 16, 1024);
    const uint64_t cols0 = sdesc_sw128(f.base + C::kRing0, kChunkBytes, 1024);
    const uint32_t tmem = f.tmem;
    bool ok = true;
    // S = Q K^T (which = 0) or dP = dO V^T (1) for stream step g, of item q
    auto issue_s = [&](int which, int q, int g) {
      const uint64_t a = res + (2 * (u32(q) % C::kResBufs) + which) * kTile;
      const uint64_t b = which ? rows1 + u32(g) % C::kStages1 * kTile : rows0 + u32(g) % C::kStages0 * kTile;
      mma_ss_depth_w<D>(tmem + (which ? C::kColDp : C::kColS), a, b, kIdS, 0u);
      mma_commit_w(f.bar(which ? C::kBarDp : C::kBarS));
    };
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const int ns = f.items()[u32(q) % kItems].ns;
      f.give_item(q);
      if (warp == kMmaWarp) {
        // S and dP, each once its predecessor is in registers (both once dP is: 668
        // us instead of 588 for the call, 8 documents of up to 4096 tokens, 32 / 8 heads)
        ok = f.resident(q);
        for (int jj = 0; jj < ns && ok; ++jj) {
          const int gs = g + jj;
          ok = (gs == 0 || f.wait(C::kBarP, gs - 1)) && f.landed0(gs) && f.ready(gs);
          if (!ok) break;
          tc_fence_after();
          issue_s(0, q, gs);
          ok = (gs == 0 || f.wait(C::kBarDpFree, gs - 1)) && f.landed1(gs);
          if (!ok) break;
          tc_fence_after();
          issue_s(1, q, gs);
          mma_commit_w(f.bar(C::kBarEmpty1 + u32(gs) % C::kStages1));
        }
        if (ok) mma_commit_w(f.bar(C::kBarResFree + u32(q) % C::kResBufs));
      } else {
        // dQ (+)= dS K; that dS is there says that S has been computed
        for (int jj = 0; jj < ns && ok; ++jj) {
          const int gs = g + jj;
          ok = f.landed0(gs) && f.ready(gs) && (jj > 0 || q == 0 || f.wait(C::kBarAccFree, q - 1)) && f.wait(C::kBarDs, gs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t b = cols0 + u32(gs) % C::kStages0 * kTile;
          mma_ts_depth_w<false>(tmem + C::kColA, tmem + C::kColDs, b, kIdA, jj > 0 ? 1u : 0u);
          mma_commit_w(f.bar(C::kBarDsFree));
          mma_commit_w(f.bar(C::kBarEmpty0 + u32(gs) % C::kStages0));
        }
        if (ok) mma_commit_w(f.bar(C::kBarFinal));
      }
      g += ns;
    }
    f.drain(warp == kMmaWarp ? 0 : 1);
  } else if (warp >= kOutWarp) {
    // ------------------------------------------------------------ write-back
    f.write_back([&](const Item& it, auto&& put) {
      const int row = (warp & 3) * 32;
      const long long stride = args.out_stride[0];
      __nv_bfloat16* out = args.out[0] + static_cast<long long>(it.row0 + it.x0) * stride + static_cast<long long>(it.h) * (G * D);
      put(0, args.scale, [&](int r) {
        const int x = sh.by_group.div(row + r);
        return x < sh.tpt && it.x0 + x < it.n ? out + x * stride + (row + r - x * G) * D : nullptr;
      });
    });
  } else {
    // ------------------------------------------------------------ dS
    regs_increase<kComputeRegs>();
    const int wg = warp / 4, r = threadIdx.x & 127, ri = sh.by_group.div(r);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int warp_i0 = sh.by_group.div(r - lane), warp_i1 = sh.by_group.div(r - lane + 31);  // tokens of the warp's rows
    const uint32_t tS = f.tmem + lane_base + C::kColS + wg * kCols;  // the group's keys are kCols wg .. kCols (wg + 1) - 1
    const uint32_t tDp = f.tmem + lane_base + C::kColDp + wg * kCols;
    const uint32_t tDs = f.tmem + lane_base + C::kColDs + wg * kCols / 2;
    const float2 sl2 = make_float2(args.scale_log2, args.scale_log2);
    bool ok = true;
    int g = 0;
    for (int q = 0; ok; ++q) {
      ok = f.get_item(q);
      if (!ok || f.items()[u32(q) % kItems].end) break;
      const Item& it = f.items()[u32(q) % kItems];
      const int ns = it.ns, n = it.n, i0 = it.x0, pos = i0 + ri;
      float l = -INFINITY, d = 0.f;
      if (ri < sh.tpt && pos < n) {
        const long long at = (static_cast<long long>(it.h) * sh.T + it.row0 + i0) * G + r;
        l = __ldcg(args.neg_lse + at);
        d = __ldcg(args.neg_d + at);
      }
      const float2 l2 = make_float2(l, l), d2 = make_float2(d, d);
      const int key_lo = sh.window > 0 ? pos - sh.window + 1 : 0;
      const int key_hi = sh.causal ? min(n, pos + 1) : n;  // exclusive
      // keys that all rows of the warp see: full_lo <= key < full_hi
      const int full_hi = sh.causal ? min(n, i0 + warp_i0 + 1) : n;
      const int full_lo = sh.window > 0 ? i0 + warp_i1 - sh.window + 1 : 0;
      int key0 = it.t0 * kKT;
      for (int jj = 0; jj < ns; ++jj, ++g, key0 += kKT) {
        ok = f.wait_calm(C::kBarS, g);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[32], pk[16];
        float2 p[16];
        tmem_ld32(tS, x);
        tmem_ld_wait(x);
        tc_fence_before();
        mbar_arrive_warp(f.bar(C::kBarP));
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 a = __ffma2_rn(pair(x + 2 * c), sl2, l2);
          p[c] = make_float2(ex2(a.x), ex2(a.y));
        }
        ok = f.wait_calm(C::kBarDp, g);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tDp, x);
        tmem_ld_wait(x);
        tc_fence_before();
        mbar_arrive_warp(f.bar(C::kBarDpFree));
        const bool cut = key0 + wg * kCols + kCols > full_hi || key0 + wg * kCols < full_lo;
#pragma unroll
        for (int c = 0; c < 16; ++c) p[c] = __fmul2_rn(p[c], __fadd2_rn(pair(x + 2 * c), d2));
        if (cut) {
          const int at = key0 + wg * kCols;
          keep_bits(p, bits_between(key_lo - at, key_hi - at));
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(p[c].x, p[c].y);
        if (g > 0) ok = f.wait_calm(C::kBarDsFree, g - 1);
        if (!ok) break;
        tc_fence_after();
        tmem_st16(tDs, pk);
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(f.bar(C::kBarDs));
      }
      if (!ok) break;
      f.give_item(q);
    }
  }
  f.close(res_loads, stage_loads, args.status);
}

// ---------------------------------------------------------------- launches
// The workspace: -LSE and -D, then the two lists where they are made.
struct BwdPlan {
  int slots;
  int cap[2], unit[2];  // dK and dV; dQ
  bool listed[2];
  size_t head[2];       // offsets
  size_t bytes;
};

BwdPlan bwd_plan(int B, int T, int Hq, int Hkv, int sms) {
  BwdPlan p;
  p.slots = sms;
  p.unit[0] = kKT;
  p.unit[1] = 128 / (Hq / Hkv);
  p.bytes = (static_cast<size_t>(T) * Hq * 8 + 255) / 256 * 256;
  for (int i = 0; i < 2; ++i) {
    p.cap[i] = T / p.unit[i] + B;
    p.listed[i] = static_cast<long long>(p.cap[i]) * Hkv > p.slots;
    p.head[i] = p.bytes;
    if (p.listed[i]) p.bytes += (sizeof(PackedHead) + static_cast<size_t>(p.cap[i]) * sizeof(int4) + 255) / 256 * 256;
  }
  return p;
}

template <int D>
int launch_d(const PackedBwd& b, const BwdPlan& plan, const PackedList (&lists)[2], float* stats, cudaStream_t stream) {
  const PackedProblem& p = b.p;
  const PackedShape& s = p.s;
  const int G = s.by_group.G;
  int* status = device_status_word();
  CUtensorMap mq, mk, mv, mo;
  if (!status || !make_map_packed(&mq, p.q, s.T, s.Hkv, G, D, p.q_stride, s.tpt) ||
      !make_map_packed(&mk, p.k, s.T, s.Hkv, 1, D, p.k_stride, kKT) ||
      !make_map_packed(&mv, p.v, s.T, s.Hkv, 1, D, p.v_stride, kKT) ||
      !make_map_packed(&mo, b.dO, s.T, s.Hkv, G, D, b.do_stride, s.tpt))
    return -3;
  const auto dkv = packed_dkv_kernel<D>;
  const auto dq = packed_dq_kernel<D>;
  // attribute slots 32 to 35 (the other kernels use 0-31)
  constexpr int kSlot = D == 64 ? 32 : 34;
  constexpr int kDkvBytes = Cfg<D, true>::kSmemBytes, kDqBytes = Cfg<D, false>::kSmemBytes;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(dkv), kDkvBytes, kSlot) ||
      !ensure_smem_attr(reinterpret_cast<const void*>(dq), kDqBytes, kSlot + 1))
    return -3;
  const bool all_own = s.window == 1;
  const long long rows = static_cast<long long>(s.T) * s.Hq, per = kSumThreads / (D / 8) * 2;
  SumArgs sum{};
  sum.s = s;
  sum.status = status;
  for (const PackedList& l : lists)
    if (l.entries != nullptr && !all_own) sum.lists[sum.n_lists++] = l;
  sum.n_own = std::min((own_items(s, all_own ? s.T : s.B) + kSumWarps - 1) / kSumWarps, device_sm_count() * 4);
  sum.q = static_cast<const __nv_bfloat16*>(p.q);
  sum.k = static_cast<const __nv_bfloat16*>(p.k);
  sum.v = static_cast<const __nv_bfloat16*>(p.v);
  sum.dq = static_cast<__nv_bfloat16*>(b.dq);
  sum.dk = static_cast<__nv_bfloat16*>(b.dk);
  sum.dv = static_cast<__nv_bfloat16*>(b.dv);
  sum.q_stride = p.q_stride;
  sum.k_stride = p.k_stride;
  sum.v_stride = p.v_stride;
  sum.dq_stride = b.dq_stride;
  sum.dk_stride = b.dk_stride;
  sum.dv_stride = b.dv_stride;
  sum.scale = p.scale;
  sum.scale_log2 = p.scale * kLog2e;
  const long long sum_blocks = (all_own ? 0 : (rows + per - 1) / per) + sum.n_lists + sum.n_own;
  cudaError_t e = launch_overlapped(packed_rowsum_kernel<D>, dim3(static_cast<unsigned>(sum_blocks)), dim3(kSumThreads), 0, stream, static_cast<const __nv_bfloat16*>(b.o),
                                    static_cast<const __nv_bfloat16*>(b.dO), b.do_stride, b.lse, stats, stats + rows,
                                    GroupDiv::of(s.Hq), rows, sum);
  if (e != cudaSuccess) return -3;
  if (all_own) return cudaGetLastError() == cudaSuccess ? 0 : -3;
  BwdArgs a{};
  a.s = s;
  a.neg_lse = stats;
  a.neg_d = stats + rows;
  a.status = status;
  a.scale = p.scale;
  a.scale_log2 = p.scale * kLog2e;  // (0 too: keys that are not seen are taken out after the exponential)
  auto grid = [&](int i) { return dim3(plan.listed[i] ? plan.slots : plan.cap[i] * s.Hkv); };
  a.list = lists[0];
  a.out[0] = static_cast<__nv_bfloat16*>(b.dk);
  a.out[1] = static_cast<__nv_bfloat16*>(b.dv);
  a.out_stride[0] = b.dk_stride;
  a.out_stride[1] = b.dv_stride;
  e = launch_overlapped(dkv, grid(0), dim3(kThreads), kDkvBytes, stream, mk, mv, mq, mo, a);
  if (e != cudaSuccess) return -3;
  a.list = lists[1];
  a.out[0] = static_cast<__nv_bfloat16*>(b.dq);
  a.out_stride[0] = b.dq_stride;
  e = launch_overlapped(dq, grid(1), dim3(kThreads), kDqBytes, stream, mq, mo, mk, mv, a);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace

size_t packed_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int sms) { return bwd_plan(B, T, Hq, Hkv, sms).bytes; }

int launch_packed_bwd(const PackedBwd& b, void* workspace, cudaStream_t stream) {
  const PackedShape& s = b.p.s;
  const int sms = device_sm_count();
  if (sms <= 0) return -3;
  const BwdPlan plan = bwd_plan(s.B, s.T, s.Hq, s.Hkv, sms);
  PackedList lists[2];
  for (int i = 0; i < 2; ++i) {
    lists[i] = PackedList{nullptr, nullptr, plan.cap[i], plan.unit[i], 2, i == 0 ? 1 : 0};
    if (plan.listed[i]) {
      lists[i].head = reinterpret_cast<PackedHead*>(static_cast<char*>(workspace) + plan.head[i]);
      lists[i].entries = reinterpret_cast<int4*>(lists[i].head + 1);
    }
  }
  float* stats = static_cast<float*>(workspace);
  return b.p.d == 64 ? launch_d<64>(b, plan, lists, stats, stream) : launch_d<128>(b, plan, lists, stats, stream);
}

}  // namespace fa
