// Attention over a paged e4m3 cache for many query rows (chunks of a prompt,
// whole prompts), on the tensor cores through tensor memory.
//
// Mathematics as in fa_paged_attn.cu: numerators relative to the maximum of
// s_j + log2 sv_j, denominators relative to the maximum of s_j, cached codes
// as f16 operands. The loop is the forward's (fa_fwd.cu: query tiles resident,
// key tiles streamed, P over S in tensor memory, references that move only
// when passed by 2^8); what is new is where the operands come from.
//
// What bounds it: 4 d flops per visible (row, key) pair, on the tensor core,
// with one exponential per pair beside them. The tensor core reads its
// operands from shared memory as f16, so the codes are widened on the way: a
// TMA warp fetches a tile's codes (128 keys, 16 KiB of K and of V at d = 128),
// four warps widen them into the 128-byte-swizzled layout that the matrix
// descriptors name, and the MMA warp takes them from there. Widening costs
// about 300 instructions per thread and tile, next to the 256 rows that
// share the tile; doing it once per pair of 128-row tiles is why a CTA holds
// two of them.
//
// Scales within a tile. A tile of 128 keys touches up to eight pages with
// scales of their own. Widened codes are multiplied by the ratio of their
// page's scale to the tile's largest, a power of two of 2^-8 or more, which
// is exact in f16, so the softmax sees one scale per tile and costs no more
// than without scales. Tiles whose scales are further apart, or are no powers
// of two, keep their codes as they are and take a softmax that applies the
// scales group by group (16 keys) and computes numerators and denominators
// apart.
//
// Rows are packed: row r of a sequence and key head is query r / G, head r % G
// of the group, so that a group's heads share the key tiles.
//
// CTA organisation (512 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax of query tiles 0 and 1 (thread = row = TMEM lane)
//   warps 8-11      widening
//   warp 12         MMA issue and TMEM allocation
//   warp 13         TMA producer, page and scale lookup
//   warps 14, 15    none (they complete the warpgroup that gives registers up)

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;         // query rows per tile
constexpr int kBN = 128;         // keys per tile
constexpr int kThreads = 512;
constexpr int kWidenWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr int kGroups = kBN / 16;
constexpr int kInfos = 8;        // tiles' scale records kept
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;    // log2 units that a weight may pass its reference by
constexpr float kPShift = 6.f;   // P is held as 2^6 P

// What the softmax and the widening need to know of a tile.
struct TileInfo {
  float ek;               // 2^(largest exponent of the keys' scales)
  float ev;               // log2 of the values' largest scale (its exponent)
  int by_group;           // 1: scales applied group by group
  int absent;             // 1: some group of 16 keys has no page to read
  uint32_t kh[kGroups];   // what a group's widened codes are multiplied by (f16 pair): scale / largest
  uint32_t vh[kGroups];
  float kr[kGroups];      // by_group: the keys' scale relative to ek (below 0: group absent)
  float vr[kGroups];      // and log2 of the values' scale
};

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kBN * 128;              // 128 rows x 64 f16
  static constexpr int kTileBytes = kChunks * kChunkBytes;   // widened
  static constexpr int kRawBytes = kBN * D;                  // codes
  static constexpr int kStages = 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kRawKOff = kVOff + kStages * kTileBytes;
  static constexpr int kRawVOff = kRawKOff + kRawBytes;
  static constexpr int kInfoOff = kRawVOff + kRawBytes;
  static constexpr int kBarOff = kInfoOff + kInfos * static_cast<int>(sizeof(TileInfo));
  enum : int {
    kBarQFull = 0,
    kBarRawKFull, kBarRawKEmpty, kBarRawVFull, kBarRawVEmpty,
    kBarKFull,                          // two of each from here
    kBarKEmpty = kBarKFull + kStages,
    kBarVFull = kBarKEmpty + kStages,
    kBarVEmpty = kBarVFull + kStages,
    kBarSFull = kBarVEmpty + kStages,
    kBarPFull = kBarSFull + 2,
    kBarOFinal = kBarPFull + 2,
    kBarDrain = kBarOFinal + 2,
    kNumBars
  };
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;  // + slack to align the base
  static constexpr uint32_t kColO = 2 * kBN;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColO + 2 * D <= kTmemCols, "accumulators exceed tensor memory");
  static_assert(kSmemBytes <= 232448, "tiles exceed shared memory");
};

struct ChunkArgs {
  PagedBatchDev batch;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;
  float* lse;
  const uint8_t* v_pages;
  const float* k_scales;
  const float* v_scales;
  int* status;
  int Hq, Hkv, G;
  int window;
  int pairs;         // of 256 rows: those of the longest packed sequence and a key head
  float scale_log2;
};

__device__ __forceinline__ int exponent_of(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;  // of a positive normal number
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const ChunkArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_u32);
  auto bar = [&](int i) -> uint32_t { return base + C::kBarOff + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  volatile int* nan_flag = abort_flag + 1;
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    mbar_init(bar(C::kBarQFull), 8);
    mbar_init(bar(C::kBarRawKFull), 1);
    mbar_init(bar(C::kBarRawKEmpty), 4);
    mbar_init(bar(C::kBarRawVFull), 1);
    mbar_init(bar(C::kBarRawVEmpty), 4);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarKFull + s), 4);
      mbar_init(bar(C::kBarKEmpty + s), 1);
      mbar_init(bar(C::kBarVFull + s), 4);
      mbar_init(bar(C::kBarVEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      // the MMAs' completion, and the MMA warp itself, which passes on that
      // the tile's records (and, at the end, the NaN flag) have been written
      mbar_init(bar(C::kBarSFull + t), 2);
      mbar_init(bar(C::kBarPFull + t), 4);
      mbar_init(bar(C::kBarOFinal + t), 2);
    }
    mbar_init(bar(C::kBarDrain), 1);
    *abort_flag = 0;
    *nan_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();

  // The item: heaviest (last) pairs of rows first.
  const int per_pair = a.batch.B * a.Hkv;
  const int pair = a.pairs - 1 - static_cast<int>(blockIdx.x / per_pair);
  const int h = static_cast<int>(blockIdx.x % per_pair) % a.Hkv;
  const int seq = static_cast<int>(blockIdx.x % per_pair) / a.Hkv;
  const PagedSeq s = paged_seq(a.batch, seq, a.status);
  const int rows = s.n * a.G, p0 = s.len - s.n;
  int r0[2], lo_t[2], n_t[2], p_first[2], p_last[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    r0[t] = pair * 2 * kBM + t * kBM;
    p_first[t] = p0 + r0[t] / a.G;
    p_last[t] = p0 + (min(r0[t] + kBM, rows) - 1) / a.G;
    const int hi = r0[t] < rows && p_last[t] >= 0 ? p_last[t] / kBN + 1 : 0;
    lo_t[t] = a.window > 0 ? max(p_first[t] - a.window + 1, 0) / kBN : 0;
    n_t[t] = max(hi - lo_t[t], 0);
  }
  const int j_first = n_t[0] == 0 ? lo_t[1] : n_t[1] == 0 ? lo_t[0] : min(lo_t[0], lo_t[1]);
  const int j_end = max(n_t[0] > 0 ? lo_t[0] + n_t[0] : 0, n_t[1] > 0 ? lo_t[1] + n_t[1] : 0);
  const int n_stream = max(j_end - j_first, 0);
  const int a0 = lo_t[0] - j_first, b0 = a0 + n_t[0], a1 = lo_t[1] - j_first, b1 = a1 + n_t[1];
  // keys that every row of the CTA sees lie in [full_lo, full_hi]
  const int full_hi = p_first[0];
  const int full_lo = a.window > 0 ? (r0[1] < rows ? p_last[1] : p_last[0]) - a.window + 1 : 0;
  // keys that any row sees lie in [key_lo, key_end)
  const int key_lo = a.window > 0 ? max(p_first[0] - a.window + 1, 0) : 0;
  const int key_end = max(max(p_last[0], r0[1] < rows ? p_last[1] : 0) + 1, 0);

  if (warp >= kMmaWarp) {
    regs_decrease<56>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- TMA warp
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
      // Lane i looks up the i-th of 32 groups of 16 keys (four tiles): its
      // page, then its scales. The next four tiles' loads are under way while
      // the present ones are issued.
      const int box_rows = min(a.batch.page_size, kBN), boxes = kBN / box_rows, per_box = box_rows / 16;
      int n_page = -1;
      float n_sk = 1.f, n_sv = 1.f;
      bool n_want = false;
      auto look = [&](int step) {
        const int j0 = (j_first + step) * kBN + lane * 16;
        n_want = step + (lane >> 3) < n_stream && j0 < key_end && j0 + 16 > key_lo;
        n_page = n_want ? paged_page(a.batch, seq, j0 >> a.batch.page_shift, a.status) : -1;
      };
      auto scales = [&]() {
        n_sk = n_sv = 1.f;
        if (n_page >= 0) {
          const long long at = static_cast<long long>(n_page) * a.Hkv + h;
          n_sk = a.k_scales[at];
          n_sv = a.v_scales[at];
        }
      };
      bool ok = true;
      int k_copies = 0, v_copies = 0;
      look(0);
      scales();
      for (int base4 = 0; base4 < n_stream && ok; base4 += 4) {
        const int page = n_page;
        const float sk = n_sk, sv = n_sv;
        const bool on = page >= 0, missing = n_want && !on;
        look(base4 + 4);
        // the four tiles' scales, eight lanes each
        const bool pow2 = (__float_as_uint(sk) & 0x7fffffu) == 0 && (__float_as_uint(sv) & 0x7fffffu) == 0 &&
                          sk > 0.f && sv > 0.f && sk < INFINITY && sv < INFINITY;
        const int ke = on ? exponent_of(sk) : -1000, ve = on ? exponent_of(sv) : -1000;
        int kmax = ke, vmax = ve, kmin = on ? ke : 1000, vmin = on ? ve : 1000;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
          kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, d));
          vmax = max(vmax, __shfl_xor_sync(0xffffffffu, vmax, d));
          kmin = min(kmin, __shfl_xor_sync(0xffffffffu, kmin, d));
          vmin = min(vmin, __shfl_xor_sync(0xffffffffu, vmin, d));
        }
        const uint32_t mine = 0xffu << (lane & 24);
        const bool by_group = (__ballot_sync(0xffffffffu, (on && !pow2) || missing) & mine) != 0 ||
                              kmax - kmin > 8 || vmax - vmin > 8;
        const bool absent = (__ballot_sync(0xffffffffu, !on) & mine) != 0;
        kmax = min(max(kmax, -126), 126);
        vmax = min(max(vmax, -126), 126);
        const float ek = pow2i(kmax);
        const float kh = by_group ? 1.f : on ? pow2i(ke - kmax) : 0.f, vh = by_group ? 1.f : on ? pow2i(ve - vmax) : 0.f;
        const float kr = !on ? -1.f : sk / ek, vr = log2f(sv);
        for (int i = 0; i < 4 && base4 + i < n_stream; ++i) {
          const int jj = base4 + i;
          if (i == 2) scales();
          // lane b: the page of box b of the tile
          int bp = __shfl_sync(0xffffffffu, page, 8 * i + (lane & 7) * per_box % 8);
          for (int q = 1; q < per_box; ++q) bp = max(bp, __shfl_sync(0xffffffffu, page, 8 * i + ((lane & 7) * per_box + q) % 8));
          const bool box = lane < boxes && bp >= 0;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box)) * static_cast<uint32_t>(box_rows * D);
          const int slot = (lane * box_rows) & (a.batch.page_size - 1), blk = bp * a.Hkv + h;
          if (jj >= 1) ok = mbar_wait_w(bar(C::kBarRawKEmpty), (jj - 1) & 1, abort_flag);
          if (!ok) break;
          if (box)
            tma_load_3d(base + C::kRawKOff + lane * box_rows * D, &tmK, bar(C::kBarRawKFull), 0, slot, blk);
          if ((lane >> 3) == i) {
            TileInfo& ti = infos[jj % kInfos];
            const int g = lane & 7;
            ti.kh[g] = pack_f16(kh, kh);
            ti.vh[g] = pack_f16(vh, vh);
            ti.kr[g] = kr;
            ti.vr[g] = vr;
            if (g == 0) {
              ti.ek = ek;
              ti.ev = static_cast<float>(vmax);
              ti.by_group = by_group ? 1 : 0;
              ti.absent = absent ? 1 : 0;
            }
          }
          __syncwarp();
          // (bytes that have landed already count as well: the phase cannot end before this arrival)
          if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarRawKFull), bytes);
          ++k_copies;
          if (jj >= 1) ok = mbar_wait_w(bar(C::kBarRawVEmpty), (jj - 1) & 1, abort_flag);
          if (!ok) break;
          if (box)
            tma_load_3d(base + C::kRawVOff + lane * box_rows * D, &tmV, bar(C::kBarRawVFull), 0, slot, blk);
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarRawVFull), bytes);
          ++v_copies;
        }
        if (base4 + 2 >= n_stream) break;  // (fewer than three tiles in this batch: none follows)
      }
      // Let the copies in flight land before the CTA can end, whoever gives up:
      // each buffer's last phase (over already unless someone did).
      if (k_copies > 0) mbar_wait(bar(C::kBarRawKFull), (k_copies - 1) & 1, nullptr);
      if (v_copies > 0) mbar_wait(bar(C::kBarRawVFull), (v_copies - 1) & 1, nullptr);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t kIdS = idesc_f16_f32(kBM, kBN, false, false);
      constexpr uint32_t kIdO = idesc_f16_f32(kBM, D, false, true);
      bool ok = n_stream > 0 ? mbar_wait_w(bar(C::kBarQFull), 0, abort_flag) : false;
      tc_fence_after();
      int k_ready = -1;
      auto ensure_k = [&](int jj) {
        if (ok && jj > k_ready) {
          ok = mbar_wait_w(bar(C::kBarKFull + jj % C::kStages), (jj / C::kStages) & 1, abort_flag);
          tc_fence_after();
          k_ready = jj;
        }
      };
      const uint64_t dQ0 = sdesc_sw128(base + C::kQOff, 16, 1024);
      const uint64_t dK0 = sdesc_sw128(base + C::kKOff, 16, 1024);
      const uint64_t dV0 = sdesc_sw128(base + C::kVOff, C::kChunkBytes, 1024);
      auto issue_s = [&](int t, int jj) {
        const uint64_t q = dQ0 + static_cast<uint64_t>(t * C::kTileBytes >> 4);
        const uint64_t k = dK0 + static_cast<uint64_t>((jj % C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4);
          mma_ss_w(tmem + t * kBN, q + off, k + off, kIdS, kk > 0 ? 1u : 0u);
        }
        mma_commit_w(bar(C::kBarSFull + t));
        mbar_arrive_warp(bar(C::kBarSFull + t));
      };
      auto issue_pv = [&](int t, int jj, bool first) {
        const uint64_t v = dV0 + static_cast<uint64_t>((jj % C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          mma_ts_w(tmem + C::kColO + t * D, tmem + t * kBN + kk * 8, v + 128 * kk, kIdO,
                   (!first || kk > 0) ? 1u : 0u);
      };
      auto step_of = [&](int t, int jj) -> int {  // tile-local step, or -1
        const int x = t == 0 ? a0 : a1, y = t == 0 ? b0 : b1;
        return (jj >= x && jj < y) ? jj - x : -1;
      };
      // P overwrites S: each tile's next QK^T is issued after its P.V. Step
      // jj: per tile, the P.V of key tile jj, then the QK^T of jj + 1 (the
      // first step, -1, has none of the former). One copy of the code for
      // both tiles: the loops of the four roles share the instruction cache.
#pragma unroll 1
      for (int jj = -1; jj < n_stream && ok; ++jj) {
        if (jj >= 0) {
          ok = mbar_wait_w(bar(C::kBarVFull + jj % C::kStages), (jj / C::kStages) & 1, abort_flag);
          tc_fence_after();
        }
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int u = step_of(t, jj);
          if (ok && u >= 0) {
            ok = mbar_wait_w(bar(C::kBarPFull + t), u & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, jj, u == 0);
            if (jj + 1 >= (t == 0 ? b0 : b1)) {
              mma_commit_w(bar(C::kBarOFinal + t));
              mbar_arrive_warp(bar(C::kBarOFinal + t));
            }
          }
          if (ok && step_of(t, jj + 1) >= 0) {
            ensure_k(jj + 1);
            if (!ok) break;
            issue_s(t, jj + 1);
          }
        }
        if (!ok) break;
        if (jj >= 0) mma_commit_w(bar(C::kBarVEmpty + jj % C::kStages));
        if (jj + 1 < n_stream) mma_commit_w(bar(C::kBarKEmpty + (jj + 1) % C::kStages));
      }
      // let every MMA this warp issued finish before TMEM is released
      mma_commit_w(bar(C::kBarDrain));
      mbar_wait_w(bar(C::kBarDrain), 0, nullptr);
    }
  } else if (warp >= kWidenWarp) {
    regs_decrease<88>();
    // ------------------------------------------------------------ widening
    // Eight codes per thread and step become one 16-byte unit of the widened
    // row. The eight lanes of a store phase hold the eight units of one row,
    // which the swizzle spreads over all banks; a thread's rows are 16 apart,
    // so its swizzle and all offsets are fixed.
    const int tid = threadIdx.x - 32 * kWidenWarp;
    const int unit = tid & 7, row0 = tid >> 3;
    constexpr int kSteps = kBN / 16;
    const uint32_t src0 = static_cast<uint32_t>(row0 * D + unit * 8);
    const uint32_t dst0 = static_cast<uint32_t>(row0 * 128 + ((unit ^ (row0 & 7)) << 4));
    bool ok = true;
    bool saw_nan = false;
#pragma unroll 1
    for (int w2 = 0; w2 < 2 * n_stream && ok; ++w2) {  // keys and values in turn
      const int jj = w2 >> 1, st = jj % C::kStages;
      const bool values = w2 & 1;
      const TileInfo& ti = infos[jj % kInfos];
      const int key0 = (j_first + jj) * kBN;
      const uint8_t* raw = smem + (values ? C::kRawVOff : C::kRawKOff) + src0;
      uint8_t* out = smem + (values ? C::kVOff : C::kKOff) + st * C::kTileBytes + dst0;
      ok = mbar_wait_w(bar(values ? C::kBarRawVFull : C::kBarRawKFull), jj & 1, abort_flag);
      if (ok && jj >= C::kStages)
        ok = mbar_wait_w(bar((values ? C::kBarVEmpty : C::kBarKEmpty) + st), ((jj / C::kStages) + 1) & 1, abort_flag);
      if (!ok) break;
      const uint32_t* ratios = values ? ti.vh : ti.kh;
      // Values of keys that some row does not see: 0 x NaN is NaN, so no code
      // of theirs may be one. Groups without a page: nothing was loaded.
      const bool check = ti.absent || (values && (key0 + kBN - 1 > full_hi || key0 < full_lo));
      // Codes are fetched eight units ahead of the stores: the compiler cannot
      // move a shared load above a shared store itself, and one unit at a time
      // is all latency (115 cycles each, against about 12 instructions).
      constexpr int kUnits = kSteps * C::kChunks, kBatch = 8;
      uint2 w[kUnits];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        w[i] = *reinterpret_cast<const uint2*>(raw + i / C::kChunks * 16 * D + i % C::kChunks * 64);
#pragma unroll
      for (int b = 0; b < kUnits; b += kBatch) {
        if (b + kBatch < kUnits) {
#pragma unroll
          for (int i = b + kBatch; i < b + 2 * kBatch; ++i)
            w[i] = *reinterpret_cast<const uint2*>(raw + i / C::kChunks * 16 * D + i % C::kChunks * 64);
        }
        uint32_t ratio[kBatch / C::kChunks];
#pragma unroll
        for (int i = 0; i < kBatch / C::kChunks; ++i) ratio[i] = ratios[b / C::kChunks + i];
        if (check) {
#pragma unroll
          for (int i = b; i < b + kBatch; ++i) {
            const int g = i / C::kChunks;
            if (ti.kr[g] < 0.f) w[i] = make_uint2(0, 0);
            if (values && (key0 + g * 16 + 15 > full_hi || key0 + g * 16 < full_lo)) {
              const uint2 z = make_uint2(nan_bytes(w[i].x), nan_bytes(w[i].y));
              saw_nan = saw_nan || (z.x | z.y) != 0;
              w[i] = make_uint2(w[i].x & ~z.x, w[i].y & ~z.y);
            }
          }
        }
#pragma unroll
        for (int i = b; i < b + kBatch; ++i) {
          const uint32_t r = ratio[(i - b) / C::kChunks];
          *reinterpret_cast<uint4*>(out + i / C::kChunks * 2048 + i % C::kChunks * C::kChunkBytes) =
              make_uint4(hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].x)), r),
                         hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].x >> 16)), r),
                         hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].y)), r),
                         hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i].y >> 16)), r));
        }
      }
      if (saw_nan) *nan_flag = 1;
      fence_async_smem();
      mbar_arrive_warp(bar((values ? C::kBarVFull : C::kBarKFull) + st));
      mbar_arrive_warp(bar(values ? C::kBarRawVEmpty : C::kBarRawKEmpty));
    }
  } else {
    regs_increase<184>();
    // ------------------------------------------------------------ softmax
    const int t = warp / 4;
    const int n_mine = n_t[t], row0_tile = r0[t];
    const int step0 = t == 0 ? a0 : a1;
    const int r = row0_tile + (threadIdx.x & 127);  // packed row
    const bool live = r < rows;
    const int i = live ? r / a.G : 0, hd = h * a.G + (live ? r % a.G : 0);
    const int p = live ? p0 + i : p_last[t];
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * kBN;
    const uint32_t tO = tmem + lane_base + C::kColO + t * D;
    uint8_t* q_tile = smem + C::kQOff + t * C::kTileBytes;
    float qf = 0.f;
    if (n_stream > 0) {
      // this row's query, scaled into f16 by a power of two (exact within 2^27 of its largest value)
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(s.row0 + i) * a.q_stride + hd * D);
      uint4 w[D / 8];
      float m = 0.f;
#pragma unroll
      for (int u = 0; u < D / 8; ++u) {
        w[u] = live ? src[u] : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          m = max3(m, fabsf(__uint_as_float(x[q] << 16)), fabsf(__uint_as_float(x[q] & 0xffff0000u)));
      }
      int k = 13 - exponent_of(m);
      k = m == 0.f ? 0 : min(max(k, -126), 126);
      const float up = pow2i(k);
      qf = a.scale_log2 * pow2i(-k);
#pragma unroll
      for (int u = 0; u < D / 8; ++u) {
        const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        uint32_t f[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f[q] = pack_f16(__uint_as_float(x[q] << 16) * up, __uint_as_float(x[q] & 0xffff0000u) * up);
        const int tr = threadIdx.x & 127;
        *reinterpret_cast<uint4*>(q_tile + (u >> 3) * C::kChunkBytes + tr * 128 + (((u & 7) ^ (tr & 7)) << 4)) =
            make_uint4(f[0], f[1], f[2], f[3]);
      }
      fence_async_smem();
      mbar_arrive_warp(bar(C::kBarQFull));
    }

    float ms = -INFINITY, mt = -INFINITY, l = 0.f;  // references (log2 units) and denominator
    bool ok = true;
    for (int u = 0; u < n_mine; ++u) {
      const int key0 = (j_first + step0 + u) * kBN;
      ok = mbar_wait_w(bar(C::kBarSFull + t), u & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const TileInfo& ti = infos[(step0 + u) % kInfos];
      uint32_t sr[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
      const float sl2 = qf * ti.ek, ev = ti.ev;
      const bool by_group = ti.by_group != 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
      float x[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c >> 5][c & 31]);
      if (key0 + kBN - 1 > p_first[t] || (a.window > 0 && key0 <= p_last[t] - a.window)) {
        const int lim_hi = p + 1 - key0, lim_lo = a.window > 0 ? p - a.window + 1 - key0 : 0;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= lim_hi || c < lim_lo) x[c] = -INFINITY;
      }
      const float m_tile = max3(fmaxf(max32(x), max32(x + 32)), max32(x + 64), max32(x + 96)) * sl2;
      const float ms_old = ms, mt_old = mt;
      bool moved = m_tile > fminf(ms, mt - ev) + kSlack;
      if (moved && !by_group) {
        ms = fmaxf(ms, m_tile);
        mt = fmaxf(mt, m_tile + ev);
      }
      float su = ms == -INFINITY ? 0.f : ms, tu = mt == -INFINITY ? 0.f : mt;
      // P = 2^(x sl2 + ev - m_t + 6); the denominator's terms are P 2^(m_t - ev - 6 - m_s),
      // unless the two references lie too far apart for P not to underflow
      if (!by_group && !__any_sync(0xffffffffu, su + ev - tu < -60.f)) {
        const float add = ev - tu + kPShift;
        const float2 sl2x2 = make_float2(sl2, sl2), add2 = make_float2(add, add);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 e2 = __ffma2_rn(make_float2(x[64 * hf + 2 * c], x[64 * hf + 2 * c + 1]), sl2x2, add2);
            const float2 pr = make_float2(ex2(e2.x), ex2(e2.y));
            if (c & 1) acc1 = __fadd2_rn(acc1, pr);
            else acc0 = __fadd2_rn(acc0, pr);
            pk[c] = pack_f16(pr.x, pr.y);
          }
          tmem_st32(tS + 32 * hf, pk);
        }
        const float als = moved ? ex2(ms_old - su) : 1.f;
        l = fmaf(l, als, ((acc0.x + acc0.y) + (acc1.x + acc1.y)) * ex2(tu - ev - kPShift - su));
      } else {
        // Group by group from tensor memory again, with the group's scales,
        // numerators and denominators apart. P of group g takes columns
        // 8 g .. 8 g + 7, which no later group's S lies in.
        auto group = [&](int g, float (&y)[16], float* vlog) {
          uint32_t w[16];
          tmem_ld16(tS + 16 * g, w);
          tmem_ld_wait(w);
          const float kr = by_group ? ti.kr[g] : 1.f;
          *vlog = by_group ? ti.vr[g] : ev;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int j = key0 + 16 * g + c;
            // (no page: no key of the group takes part)
            y[c] = kr >= 0.f && sees(p, j, a.window) ? __uint_as_float(w[c]) * (sl2 * kr) : -INFINITY;
          }
        };
        float vlog;
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          float y[16], m = -INFINITY;
          group(g, y, &vlog);
#pragma unroll
          for (int c = 0; c < 16; ++c) m = fmaxf(m, y[c]);
          ms = fmaxf(ms, m);
          mt = fmaxf(mt, m + vlog);
        }
        moved = true;
        su = ms == -INFINITY ? 0.f : ms;
        tu = mt == -INFINITY ? 0.f : mt;
        l *= ex2(ms_old - su);
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          float y[16];
          uint32_t pk[8];
          group(g, y, &vlog);
          const float add = vlog - tu + kPShift;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            l += ex2(y[2 * c] - su) + ex2(y[2 * c + 1] - su);
            pk[c] = pack_f16(ex2(y[2 * c] + add), ex2(y[2 * c + 1] + add));
          }
          tmem_st8(tS + 8 * g, pk);
        }
      }
      const float alpha = moved ? ex2(mt_old - tu) : 1.f;  // of the accumulator
      // O is settled: this tile's S was committed after the previous P.V
      if (u > 0 && __any_sync(0xffffffffu, moved)) {
        const float2 al2 = make_float2(alpha, alpha);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), al2);
            o[e] = __float_as_uint(v.x);
            o[e + 1] = __float_as_uint(v.y);
          }
          tmem_st32(tO + c * 32, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(bar(C::kBarPFull + t));
    }
    if (ok && row0_tile < rows) {
      const long long at = static_cast<long long>(s.row0 + i) * a.Hq + hd;
      if (n_mine > 0) ok = mbar_wait_w(bar(C::kBarOFinal + t), 0, abort_flag);
      if (ok && n_mine == 0) {
        if (live) {  // no row of the tile sees a key
          uint4* dst = reinterpret_cast<uint4*>(a.o + at * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
          a.lse[at] = -INFINITY;
        }
      } else if (ok) {
        tc_fence_after();
        const float su = ms == -INFINITY ? 0.f : ms, tu = mt == -INFINITY ? 0.f : mt;
        const float f = l == 0.f ? 0.f : ex2(tu - su - kPShift) / l;
        // as in the forward: 32 rows x 64 columns at a time through this
        // warp's part of the Q tile (free by now), so that rows leave as whole lines
        uint8_t* blk = q_tile + (warp & 3) * 4096;
        uint8_t* mine = blk + lane * 128;
#pragma unroll 1
        for (int hh = 0; hh < D / 64; ++hh) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + hh * 64 + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                w[q] = pack_bf16(__uint_as_float(o[8 * e + 2 * q]) * f, __uint_as_float(o[8 * e + 2 * q + 1]) * f);
              *reinterpret_cast<uint4*>(mine + (((4 * c + e) ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rr = 4 * j + (lane >> 3), v = lane & 7;
            const uint4 val = *reinterpret_cast<const uint4*>(blk + rr * 128 + ((v ^ (rr & 7)) * 16));
            const int pr = row0_tile + (warp & 3) * 32 + rr;
            if (pr < rows)
              *reinterpret_cast<uint4*>(a.o + (static_cast<long long>(s.row0 + pr / a.G) * a.Hq + h * a.G + pr % a.G) * D +
                                        hh * 64 + v * 8) = val;
          }
          __syncwarp();
        }
        if (live) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (su + log2f(l));
        if (*nan_flag && live) {
          // a NaN code was taken out of a tile that not every row sees: put it into the rows that do
#pragma unroll 1
          for (int j = max(a.window > 0 ? p - a.window + 1 : 0, 0); j <= p; ++j) {
            const int j0 = j & ~15;
            if (j0 + 15 <= full_hi && j0 >= full_lo) continue;
            const int page = paged_page(a.batch, seq, j >> a.batch.page_shift, a.status);
            if (page < 0) continue;
            const uint8_t* code = a.v_pages + ((static_cast<long long>(page) * a.Hkv + h) * a.batch.page_size +
                                               (j & (a.batch.page_size - 1))) * D;
#pragma unroll 1
            for (int c = 0; c < D; ++c)
              if ((code[c] & 0x7f) == 0x7f) a.o[at * D + c] = __float2bfloat16(__int_as_float(0x7fffffff));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) *a.status = kStatusTimeout;
}

template <int D>
int launch_chunk_d(const PagedPool& pool, const ChunkArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap mk, mv;
  const int blocks = pool.num_pages * pool.num_heads;
  if (!make_map_pages(&mk, pool.k_pages, blocks, pool.page_size, D, pool.page_size, false) ||
      !make_map_pages(&mv, pool.v_pages, blocks, pool.page_size, D, pool.page_size, false))
    return -3;
  auto kern = paged_chunk_kernel<D>;
  // attribute slots 28, 29
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, D == 64 ? 28 : 29)) return -3;
  const long long grid = static_cast<long long>(a.pairs) * a.batch.B * a.Hkv;
  if (grid > 0x7fffffffLL) return -1;
  const cudaError_t e = launch_overlapped(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), C::kSmemBytes,
                                          stream, mk, mv, a);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace

int launch_paged_chunk(const PagedPool& pool, const PagedBatchDev& batch, const PagedAttn& p, cudaStream_t stream) {
  ChunkArgs a{};
  a.batch = batch;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.q_stride = p.q_stride;
  a.o = static_cast<__nv_bfloat16*>(p.o);
  a.lse = p.lse;
  a.v_pages = static_cast<const uint8_t*>(pool.v_pages);
  a.k_scales = pool.k_scales;
  a.v_scales = pool.v_scales;
  a.status = device_status_word();
  if (!a.status) return -3;
  a.Hq = p.Hq;
  a.Hkv = pool.num_heads;
  a.G = p.Hq / pool.num_heads;
  a.window = p.window;
  a.pairs = static_cast<int>((static_cast<long long>(batch.max_q) * a.G + 2 * kBM - 1) / (2 * kBM));
  // scale 0 (uniform weights) runs as a tiny positive scale, as in the forward
  const float sl2 = p.scale * kLog2e;
  a.scale_log2 = sl2 > 1e-30f ? sl2 : 1e-30f;
  return pool.d == 64 ? launch_chunk_d<64>(pool, a, stream) : launch_chunk_d<128>(pool, a, stream);
}

}  // namespace fa
