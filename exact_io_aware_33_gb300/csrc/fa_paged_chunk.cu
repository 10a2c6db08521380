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
// about 200 instructions per thread for a tile of K or of V, next to the 256
// rows that share it; doing it once per pair of 128-row tiles is why a CTA
// holds two of them. Measured: 2 x 2048 queries over 8192 keys, 32 query and 8
// key heads, d = 128, in 375 us: 1.28 PFLOP/s, 67 % of the measured matrix
// product's rate. A step of a tile is 1980 cycles of softmax, then 1190 until
// the next S is there (its P.V, the next QK^T, the other tile's before them).
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
// Division of the work. An item is one sequence, key head and pair of query
// tiles (256 rows); its steps are the key tiles that any of its rows sees. As
// in fa_paged_attn.cu the steps of all items, laid end to end, are cut into
// equal parts, one per CTA, of which each SM has one for the whole call: items
// number a few per SM and their lengths differ, so whole items would leave
// SMs idle at the end (512 items on 152 SMs: four rounds instead of 3.4).
// Pieces of items go to the workspace, normalised, and a second kernel joins
// them. The TMA warp walks the part and leaves a record of each piece for the
// other warps, whose rings run on from piece to piece.
//
// CTA organisation (512 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax of query tiles 0 and 1 (thread = row = TMEM lane)
//   warps 8-11      widening
//   warp 12         MMA issue and TMEM allocation
//   warp 13         TMA producer, walk, page and scale lookup
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
constexpr int kPieces = 4;       // pieces' records kept
// An item costs about this many steps more than it has: its queries, the start
// of its chain, its write-back. Four prompts of 2048 tokens, 32 query and 8 key
// heads, d = 128: 176 us with 4, 179 with 6; 16 heads, d = 64: 80 us with 3, 83
// with 2, 82 with 4.
template <int D>
constexpr int kItemSteps = D == 64 ? 3 : 4;
constexpr int kPartSteps = 8;    // a part has at least this many
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;    // log2 units that a weight may pass its reference by
constexpr float kPShift = 6.f;   // P is held as 2^6 P
// Least factor of S: keeps -infinity, where a key is not seen, from meeting a
// factor that underflowed to 0. |S| stays below 2^37, so it changes nothing.
constexpr float kLeast = 1e-37f;

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

// A piece of an item, left by the TMA warp.
struct Piece {
  int end;               // 1: no more pieces (the rest is not set)
  int h, row0, rows;     // key head; packed rows of the sequence: first token row, and their number
  int p0, r0;            // position of query 0; first packed row of the item
  int key0, steps;       // first key, and number of key tiles
  int a0, b0, a1, b1;    // steps that query tiles 0 and 1 take part in
  int full_lo, full_hi;  // keys that every row of the item sees
  int seen_hi;           // last key that any does
  int whole;             // 1: all of the item
  int slot;              // workspace slot of a piece that is not
  int seq;
};

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kBN * 128;              // 128 rows x 64 f16
  static constexpr int kTileBytes = kChunks * kChunkBytes;   // widened
  static constexpr int kRawBytes = kBN * D;                  // codes
  static constexpr int kStages = 2;
  static constexpr int kRaw = D == 64 ? 4 : 1;  // tiles of codes ahead of the widening: as many as there is room for
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kRawKOff = kVOff + kStages * kTileBytes;
  static constexpr int kRawVOff = kRawKOff + kRaw * kRawBytes;
  static constexpr int kInfoOff = kRawVOff + kRaw * kRawBytes;
  static constexpr int kPieceOff = kInfoOff + kInfos * static_cast<int>(sizeof(TileInfo));
  static constexpr int kBarOff = kPieceOff + (kPieces * static_cast<int>(sizeof(Piece)) + 7) / 8 * 8;
  enum : int {
    kBarQFull = 0,                      // two
    kBarRawKFull = kBarQFull + 2,       // kRaw of each
    kBarRawKEmpty = kBarRawKFull + kRaw,
    kBarRawVFull = kBarRawKEmpty + kRaw,
    kBarRawVEmpty = kBarRawVFull + kRaw,
    kBarKFull = kBarRawVEmpty + kRaw,   // two of each from here
    kBarKEmpty = kBarKFull + kStages,
    kBarVFull = kBarKEmpty + kStages,
    kBarVEmpty = kBarVFull + kStages,
    kBarSFull = kBarVEmpty + kStages,
    kBarPFull = kBarSFull + 2,
    kBarOFinal = kBarPFull + 2,
    kBarPieceFull = kBarOFinal + 2,
    kBarPieceEmpty = kBarPieceFull + kPieces,
    kBarDrain = kBarPieceEmpty + kPieces,
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
  int Hq, Hkv;
  GroupDiv g;  // G = Hq / Hkv
  int window;
  float scale_log2;
  float* part_o;     // [part][2][256][d], normalised
  float* part_lse;   // [part][2][256], log2 units
  JoinRecord* records;  // [part]
};

// Where row r of a key head stands in o and lse: (token, query head).
__device__ __forceinline__ long long row_at(const ChunkArgs& a, int row0, int h, int r) {
  const int i = a.g.div(r);
  return static_cast<long long>(row0 + i) * a.Hq + h * a.g.G + (r - i * a.g.G);
}

// The key tiles of an item's two query tiles.
struct PairGeo {
  int lo[2], n[2];   // first key tile and number of them, per query tile
  int first, steps;  // of both together
};

__device__ __forceinline__ PairGeo pair_geo(const ChunkArgs& a, int rows, int p0, int pair) {
  PairGeo g;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r0 = (2 * pair + t) * kBM;
    const int p_last = p0 + a.g.div(min(r0 + kBM, rows) - 1);
    const int hi = r0 < rows && p_last >= 0 ? p_last / kBN + 1 : 0;
    g.lo[t] = first_seen(p0 + a.g.div(r0), a.window) / kBN;
    g.n[t] = max(hi - g.lo[t], 0);
  }
  g.first = g.n[0] == 0 ? g.lo[1] : g.n[1] == 0 ? g.lo[0] : min(g.lo[0], g.lo[1]);
  g.steps = max(max(g.n[0] > 0 ? g.lo[0] + g.n[0] : 0, g.n[1] > 0 ? g.lo[1] + g.n[1] : 0) - g.first, 0);
  return g;
}

__device__ __forceinline__ int pairs_of(int rows) { return (rows + 2 * kBM - 1) / (2 * kBM); }

// Steps of a pair alone: its two tiles' ranges overlap or adjoin.
__device__ __forceinline__ int pair_steps(const ChunkArgs& a, int rows, int p0, int pair) {
  const int r0 = pair * 2 * kBM, p_last = p0 + a.g.div(min(r0 + 2 * kBM, rows) - 1);
  const int hi = p_last >= 0 ? p_last / kBN + 1 : 0;
  const int lo = first_seen(p0 + a.g.div(r0), a.window) / kBN;
  return max(hi - lo, 0);
}

__device__ __forceinline__ long long scan_sum(long long own) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, own, m);
    if (lane_id() >= static_cast<uint32_t>(m)) own += x;
  }
  return own;
}

// The units (steps, and kExtra per item) of the sequences, by one warp.
// `lanes` lanes (a power of two) share a sequence's pairs, so that a batch of
// few sequences with many pairs does not take long.
template <int kExtra>
struct Units {
  int lanes;
  long long total;
  long long own, end;  // of sequence b0 + lane / lanes: its units, and the units up to its end

  __device__ __forceinline__ void scan(const ChunkArgs& a, int b0, long long before) {
    const int lane = static_cast<int>(lane_id()), b = b0 + lane / lanes;
    long long sum = 0;
    if (b < a.batch.B) {
      const PagedSeq s = paged_seq(a.batch, b, a.status);
      const int rows = s.n * a.g.G, pairs = pairs_of(rows);
      for (int i = lane % lanes; i < pairs; i += lanes) sum += pair_steps(a, rows, s.len - s.n, i) + kExtra;
    }
    end = scan_sum(sum * a.Hkv);
    for (int m = 1; m < lanes; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    own = sum * a.Hkv;
    end = before + __shfl_sync(0xffffffffu, end, lane | (lanes - 1));
  }
  __device__ __forceinline__ void start(const ChunkArgs& a) {
    lanes = 1;
    while (lanes < 32 && lanes * 2 * a.batch.B <= 32) lanes *= 2;
    long long before = 0;
    for (int b0 = 0; b0 < a.batch.B; b0 += 32 / lanes) {
      scan(a, b0, before);
      before = __shfl_sync(0xffffffffu, end, 31);
    }
    total = before;
  }
  // The sequence that holds unit u (below the total), and its first unit.
  __device__ __forceinline__ int find(const ChunkArgs& a, long long u, long long* first) {
    const int per = 32 / lanes;
    if (a.batch.B > per) scan(a, 0, 0);  // (otherwise as start() left it)
    for (int b0 = 0; b0 < a.batch.B; b0 += per) {
      if (b0 > 0) scan(a, b0, __shfl_sync(0xffffffffu, end, 31));
      const uint32_t past = __ballot_sync(0xffffffffu, end > u);
      if (past) {
        const int i = __ffs(past) - 1;
        *first = __shfl_sync(0xffffffffu, end - own, i);
        return b0 + i / lanes;
      }
    }
    *first = 0;  // not reached for u below the total
    return a.batch.B;
  }
};

// Parts that the units are cut into, and the first unit of part c.
__device__ __forceinline__ int parts_of(long long units, int ctas) {
  return static_cast<int>(min(static_cast<long long>(ctas), max(units / kPartSteps, 1LL)));
}
__device__ __forceinline__ long long part_start(long long units, int parts, int c) {
  return units * min(c, parts) / parts;
}

// An item, found from one of its units (all by one warp).
template <int kExtra>
struct Item {
  int seq, pair, h;
  PagedSeq s;
  PairGeo g;
  long long first;  // its first unit

  __device__ __forceinline__ long long units() const { return g.steps + kExtra; }
  __device__ __forceinline__ bool find(const ChunkArgs& a, Units<kExtra>& all, long long u) {
    long long before;
    seq = all.find(a, u, &before);
    if (seq >= a.batch.B) return false;
    pair = 0;
    s = paged_seq(a.batch, seq, a.status);
    const int rows = s.n * a.g.G, pairs = pairs_of(rows);
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const int i = i0 + static_cast<int>(lane_id());
      const long long own =
          i < pairs ? static_cast<long long>(a.Hkv) * (pair_steps(a, rows, s.len - s.n, i) + kExtra) : 0;
      const long long end = before + scan_sum(own);
      const uint32_t past = __ballot_sync(0xffffffffu, end > u);
      if (past) {
        const int k = __ffs(past) - 1;
        pair = i0 + k;
        before = __shfl_sync(0xffffffffu, end - own, k);
        break;
      }
      before = __shfl_sync(0xffffffffu, end, 31);
    }
    g = pair_geo(a, rows, s.len - s.n, pair);
    h = static_cast<int>((u - before) / units());
    first = before + h * units();
    return true;
  }
  // The next item; false past the last.
  __device__ __forceinline__ bool next(const ChunkArgs& a) {
    first += units();
    if (++h < a.Hkv) return true;
    h = 0;
    if (++pair < pairs_of(s.n * a.g.G)) {
      g = pair_geo(a, s.n * a.g.G, s.len - s.n, pair);
      return true;
    }
    pair = 0;
    do {
      if (++seq >= a.batch.B) return false;
      s = paged_seq(a.batch, seq, a.status);
    } while (s.n == 0);
    g = pair_geo(a, s.n * a.g.G, s.len - s.n, 0);
    return true;
  }
};

__device__ __forceinline__ int exponent_of(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;  // of a positive normal number
}

// The lowest n bits (none below 0, all above 31).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u;
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
  volatile int* nan_flag = abort_flag + 1;  // a NaN value code that some row sees was taken out (stays up)
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(bar(C::kBarRawKFull + s), 1);
      mbar_init(bar(C::kBarRawKEmpty + s), 4);
      mbar_init(bar(C::kBarRawVFull + s), 1);
      mbar_init(bar(C::kBarRawVEmpty + s), 4);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarKFull + s), 4);
      mbar_init(bar(C::kBarKEmpty + s), 1);
      mbar_init(bar(C::kBarVFull + s), 4);
      mbar_init(bar(C::kBarVEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::kBarQFull + t), 4);
      // the MMAs' completion, and the MMA warp itself, which passes on that
      // the tile's records (and, at the end, the NaN flag) have been written
      mbar_init(bar(C::kBarSFull + t), 2);
      mbar_init(bar(C::kBarPFull + t), 4);
      mbar_init(bar(C::kBarOFinal + t), 2);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bar(C::kBarPieceFull + i), 1);
      mbar_init(bar(C::kBarPieceEmpty + i), 13);  // the softmax, widening and MMA warps
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

  Piece* pieces = reinterpret_cast<Piece*>(smem + C::kPieceOff);
  // Hands piece number i to a consuming warp; false when the CTA gave up.
  auto get_piece = [&](int i, Piece* p) -> bool {
    if (!mbar_wait_w(bar(C::kBarPieceFull + i % kPieces), (i / kPieces) & 1, abort_flag)) return false;
    *p = pieces[i % kPieces];
    mbar_arrive_warp(bar(C::kBarPieceEmpty + i % kPieces));
    return true;
  };

  if (warp >= kMmaWarp) {
    regs_decrease<80>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- TMA warp
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
      // Lane i looks up the i-th of 32 groups of 16 keys (four tiles): its
      // page, then its scales. The next four tiles' loads are under way while
      // the present ones are issued.
      const int box_rows = min(a.batch.page_size, kBN), per_box = box_rows / 16;
      const uint32_t box_bytes = static_cast<uint32_t>(box_rows * D);
      constexpr int kExtra = kItemSteps<D>;
      Units<kExtra> all;
      all.start(a);
      const long long units = all.total;
      const int parts = parts_of(units, gridDim.x);
      long long u = part_start(units, parts, blockIdx.x);
      const long long u1 = part_start(units, parts, blockIdx.x + 1);
      bool ok = true;
      int gs = 0;   // steps so far: the rings run on
      int np = 0;   // pieces so far
      int k_copies = 0, v_copies = 0;
      auto put_piece = [&](const Piece& p) {
        if (np >= kPieces)
          ok = mbar_wait_w(bar(C::kBarPieceEmpty + np % kPieces), (np / kPieces - 1) & 1, abort_flag);
        if (!ok) return;
        if (lane == 0) {
          pieces[np % kPieces] = p;
          mbar_arrive(bar(C::kBarPieceFull + np % kPieces));
        }
        __syncwarp();
        ++np;
      };
      Item<kExtra> it;
      bool more = u < u1;
      if (more) more = it.find(a, all, u);
      JoinRecord record{};
      for (; more && ok && it.first < u1; more = it.next(a)) {
        // steps [s0, s1) of the item; one without steps belongs to the part of its first unit
        const int n = it.g.steps;
        const int s0 = static_cast<int>(max(u - it.first - kExtra, 0LL));
        const int s1 = static_cast<int>(min(max(u1 - it.first - kExtra, 0LL), static_cast<long long>(n)));
        if (n > 0 ? s1 <= s0 : it.first < u) continue;
        const int rows = it.s.n * a.g.G, p0 = it.s.len - it.s.n, h = it.h, seq = it.seq;
        const int r0 = it.pair * 2 * kBM;
        const int p_first = p0 + a.g.div(r0), p_last = p0 + a.g.div(min(r0 + 2 * kBM, rows) - 1);
        const int first_tile = it.g.first + s0, steps = s1 - s0;
        Piece pc;
        pc.end = 0;
        pc.seq = seq;
        pc.h = h;
        pc.row0 = it.s.row0;
        pc.rows = rows;
        pc.p0 = p0;
        pc.r0 = r0;
        pc.key0 = first_tile * kBN;
        pc.steps = steps;
        pc.a0 = min(max(it.g.lo[0] - first_tile, 0), steps);
        pc.b0 = max(min(it.g.lo[0] + it.g.n[0] - first_tile, steps), pc.a0);
        pc.a1 = min(max(it.g.lo[1] - first_tile, 0), steps);
        pc.b1 = max(min(it.g.lo[1] + it.g.n[1] - first_tile, steps), pc.a1);
        pc.full_hi = p_first;
        pc.seen_hi = p_last;
        pc.full_lo = first_seen(p_last, a.window);
        pc.whole = s0 == 0 && s1 == n;
        pc.slot = static_cast<int>(blockIdx.x) * 2 + (s0 == 0 ? 1 : 0);  // 0: continues an item, 1: begins one
        if (!pc.whole && s0 == 0)
          record = JoinRecord{parts_until(it.first + it.units(), units, parts, blockIdx.x), it.s.row0, h, r0, rows, {}};
        put_piece(pc);
        if (!ok) break;
        // keys that any row sees lie in [key_lo, key_end)
        const int key_lo = first_seen(p_first, a.window), key_end = max(p_last + 1, 0);
        int n_page = -1;
        float n_sk = 1.f, n_sv = 1.f;
        bool n_want = false;
        auto look = [&](int step) {
          const int j0 = (first_tile + step) * kBN + lane * 16;
          n_want = step + (lane >> 3) < steps && j0 < key_end && j0 + 16 > key_lo;
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
        look(0);
        scales();
        for (int base4 = 0; base4 < steps && ok; base4 += 4) {
          const int page = n_page;
          const float sk = n_sk, sv = n_sv;
          const bool on = page >= 0, missing = n_want && !on;
          look(base4 + 4);
          // this lane's box: its groups share a page, or have none to read
          int box_page = page;
          if (per_box > 1) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 1));
          if (per_box > 2) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 2));
          if (per_box > 4) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 4));
          const int grp = lane & 7;
          const bool issues = grp % per_box == 0 && box_page >= 0;
          const uint32_t issuers = __ballot_sync(0xffffffffu, issues);
          const int slot = (grp * 16) & (a.batch.page_size - 1), blk = box_page * a.Hkv + h;
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
          const float kh = by_group ? 1.f : on ? pow2i(ke - kmax) : 0.f;
          const float vh = by_group ? 1.f : on ? pow2i(ve - vmax) : 0.f;
          const float kr = !on ? -1.f : sk / ek, vr = log2f(sv);
          for (int i = 0; i < 4 && base4 + i < steps; ++i, ++gs) {
            if (i == 2) scales();
            const uint32_t bytes = __popc(issuers & (0xffu << (8 * i))) * box_bytes;
            const bool own = (lane >> 3) == i;
            const int rs = gs % C::kRaw;
            if (gs >= C::kRaw) ok = mbar_wait_w(bar(C::kBarRawKEmpty + rs), (gs / C::kRaw - 1) & 1, abort_flag);
            if (!ok) break;
            if (own) {
              if (issues) tma_load_3d(base + C::kRawKOff + rs * C::kRawBytes + grp * 16 * D, &tmK, bar(C::kBarRawKFull + rs), 0, slot, blk);
              TileInfo& ti = infos[gs % kInfos];
              ti.kh[grp] = pack_f16(kh, kh);
              ti.vh[grp] = pack_f16(vh, vh);
              ti.kr[grp] = kr;
              ti.vr[grp] = vr;
              if (grp == 0) {
                ti.ek = ek;
                ti.ev = static_cast<float>(vmax);
                ti.by_group = by_group ? 1 : 0;
                ti.absent = absent ? 1 : 0;
              }
            }
            __syncwarp();
            // (bytes that have landed already count as well: the phase cannot end before this arrival)
            if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarRawKFull + rs), bytes);
            ++k_copies;
#ifdef FA_TEST_SKIP_ARRIVE
            // Test-only build (never in libfa.so): a piece's last values are
            // never loaded, so the widening warps' bounded wait for them runs
            // out and the CTA winds down through the abort path.
            if (base4 + i == steps - 1) {
              ok = false;
              break;
            }
#endif
            if (gs >= C::kRaw) ok = mbar_wait_w(bar(C::kBarRawVEmpty + rs), (gs / C::kRaw - 1) & 1, abort_flag);
            if (!ok) break;
            if (own && issues)
              tma_load_3d(base + C::kRawVOff + rs * C::kRawBytes + grp * 16 * D, &tmV, bar(C::kBarRawVFull + rs), 0, slot, blk);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarRawVFull + rs), bytes);
            ++v_copies;
          }
        }
        u = max(u, it.first);  // from the next item on
      }
      if (lane == 0) a.records[blockIdx.x] = record;
      Piece last{};
      last.end = 1;
      if (ok) put_piece(last);
      // Let the copies in flight land before the CTA can end, whoever gives up:
      // each buffer's last phase (over already unless someone did).
      for (int i = max(k_copies - C::kRaw, 0); i < k_copies; ++i)
        mbar_wait(bar(C::kBarRawKFull + i % C::kRaw), (i / C::kRaw) & 1, nullptr);
      for (int i = max(v_copies - C::kRaw, 0); i < v_copies; ++i)
        mbar_wait(bar(C::kBarRawVFull + i % C::kRaw), (i / C::kRaw) & 1, nullptr);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t kIdS = idesc_f16_f32(kBM, kBN, false, false);
      constexpr uint32_t kIdO = idesc_f16_f32(kBM, D, false, true);
      bool ok = true;
      int gs0 = 0;         // ring position of the piece's first step
      int k_ready = -1;
      auto ensure_k = [&](int g) {
        if (ok && g > k_ready) {
          ok = mbar_wait_w(bar(C::kBarKFull + g % C::kStages), (g / C::kStages) & 1, abort_flag);
          tc_fence_after();
          k_ready = g;
        }
      };
      const uint64_t dQ0 = sdesc_sw128(base + C::kQOff, 16, 1024);
      const uint64_t dK0 = sdesc_sw128(base + C::kKOff, 16, 1024);
      const uint64_t dV0 = sdesc_sw128(base + C::kVOff, C::kChunkBytes, 1024);
      auto issue_s = [&](int t, int g) {
        const uint64_t q = dQ0 + static_cast<uint64_t>(t * C::kTileBytes >> 4);
        const uint64_t k = dK0 + static_cast<uint64_t>((g % C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4);
          mma_ss_w(tmem + t * kBN, q + off, k + off, kIdS, kk > 0 ? 1u : 0u);
        }
        mma_commit_w(bar(C::kBarSFull + t));
        mbar_arrive_warp(bar(C::kBarSFull + t));
      };
      auto issue_pv = [&](int t, int g, bool first) {
        const uint64_t v = dV0 + static_cast<uint64_t>((g % C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          mma_ts_w(tmem + C::kColO + t * D, tmem + t * kBN + kk * 8, v + 128 * kk, kIdO,
                   (!first || kk > 0) ? 1u : 0u);
      };
      // P overwrites S: each tile's next QK^T is issued after its P.V. Step
      // jj: per tile, the P.V of key tile jj, then the QK^T of jj + 1 (the
      // first step, -1, has none of the former). One copy of the code for
      // both tiles: the loops of the four roles share the instruction cache.
      int done0 = 0, done1 = 0;  // steps of each query tile before this piece
      int with0 = 0, with1 = 0;  // pieces that each had steps in before this one
      for (int np = 0; ok; ++np) {
        Piece pc;
        ok = get_piece(np, &pc);
        if (!ok || pc.end) break;
        const int n = pc.steps;
        if (n == 0) continue;
        const int a0 = pc.a0, b0 = pc.b0, a1 = pc.a1, b1 = pc.b1;
        auto step_of = [&](int t, int jj) -> int {  // tile-local step, or -1
          const int x = t == 0 ? a0 : a1, y = t == 0 ? b0 : b1;
          return (jj >= x && jj < y) ? jj - x : -1;
        };
#pragma unroll 1
        for (int jj = -1; jj < n && ok; ++jj) {
          const int g = gs0 + jj;
          if (jj >= 0) {
            ok = mbar_wait_w(bar(C::kBarVFull + g % C::kStages), (g / C::kStages) & 1, abort_flag);
            tc_fence_after();
          }
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int u = step_of(t, jj);
            if (ok && u >= 0) {
              ok = mbar_wait_w(bar(C::kBarPFull + t), ((t == 0 ? done0 : done1) + u) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, g, u == 0);
              if (jj + 1 >= (t == 0 ? b0 : b1)) {
                mma_commit_w(bar(C::kBarOFinal + t));
                mbar_arrive_warp(bar(C::kBarOFinal + t));
              }
            }
            if (ok && step_of(t, jj + 1) >= 0) {
              ensure_k(g + 1);
              if (ok && u < 0) {  // the tile's first step: its queries
                ok = mbar_wait_w(bar(C::kBarQFull + t), (t == 0 ? with0 : with1) & 1, abort_flag);
                tc_fence_after();
              }
              if (!ok) break;
              issue_s(t, g + 1);
            }
          }
          if (!ok) break;
          if (jj >= 0) mma_commit_w(bar(C::kBarVEmpty + g % C::kStages));
          if (jj + 1 < n) {
            ensure_k(g + 1);  // (a step that no tile takes part in)
            if (ok) mma_commit_w(bar(C::kBarKEmpty + (g + 1) % C::kStages));
          }
        }
        gs0 += n;
        done0 += b0 - a0;
        done1 += b1 - a1;
        with0 += b0 > a0;
        with1 += b1 > a1;
      }
      // let every MMA this warp issued finish before TMEM is released
      mma_commit_w(bar(C::kBarDrain));
      mbar_wait_w(bar(C::kBarDrain), 0, nullptr);
    }
  } else if (warp >= kWidenWarp) {
    regs_decrease<80>();
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
    int gs0 = 0;
    for (int np = 0; ok; ++np) {
      Piece pc;
      ok = get_piece(np, &pc);
      if (!ok || pc.end) break;
      const int full_lo = pc.full_lo, full_hi = pc.full_hi, seen_hi = pc.seen_hi;
#pragma unroll 1
      for (int w2 = 0; w2 < 2 * pc.steps && ok; ++w2) {  // keys and values in turn
        const int g = gs0 + (w2 >> 1), st = g % C::kStages, rs = g % C::kRaw;
        const bool values = w2 & 1;
        const TileInfo& ti = infos[g % kInfos];
        const int key0 = pc.key0 + (w2 >> 1) * kBN;
        uint8_t* raw = smem + (values ? C::kRawVOff : C::kRawKOff) + rs * C::kRawBytes + src0;
        uint8_t* out = smem + (values ? C::kVOff : C::kKOff) + st * C::kTileBytes + dst0;
        ok = mbar_wait_w(bar((values ? C::kBarRawVFull : C::kBarRawKFull) + rs), (g / C::kRaw) & 1, abort_flag);
        if (ok && g >= C::kStages)
          ok = mbar_wait_w(bar((values ? C::kBarVEmpty : C::kBarKEmpty) + st), ((g / C::kStages) + 1) & 1, abort_flag);
        if (!ok) break;
        const uint32_t* ratios = values ? ti.vh : ti.kh;
        if (ti.absent) {  // groups without a page: nothing was loaded
#pragma unroll 1
          for (int q = 0; q < kSteps; ++q) {
            if (ti.kr[q] >= 0.f) continue;
            for (int cb = 0; cb < C::kChunks; ++cb)
              *reinterpret_cast<uint2*>(raw + q * 16 * D + cb * 64) = make_uint2(0, 0);
          }
        }
        // Values of keys that some row does not see: 0 x NaN is NaN, so no code
        // of theirs may be one.
        bool check = values && (key0 + kBN - 1 > full_hi || key0 < full_lo);
        // Codes are fetched eight units ahead of the stores: the compiler cannot
        // move a shared load above a shared store itself, and one unit at a time
        // is all latency (115 cycles each, against about 12 instructions).
        constexpr int kUnits = kSteps * C::kChunks, kBatch = 8;
        uint2 w[kUnits];
      again:
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
          if (check) {
            uint32_t z = 0;  // the top bit of a byte that holds a NaN code
#pragma unroll
            for (int i = b; i < b + kBatch; ++i)
              z |= ((w[i].x & 0x7f7f7f7fu) + 0x01010101u) | ((w[i].y & 0x7f7f7f7fu) + 0x01010101u);
            if (z & 0x80808080u) {
              // rare: put this thread's codes right where they lie, and begin again
              check = false;
#pragma unroll 1
              for (int q = 0; q < kSteps; ++q) {
                if (key0 + q * 16 + 15 <= full_hi && key0 + q * 16 >= full_lo) continue;
#pragma unroll 1
                for (int cb = 0; cb < C::kChunks; ++cb) {
                  uint2* at = reinterpret_cast<uint2*>(raw + q * 16 * D + cb * 64);
                  const uint2 v = *at, n = make_uint2(nan_bytes(v.x), nan_bytes(v.y));
                  // (slots past a length may hold anything, and often do: no row to mend for those)
                  saw_nan = saw_nan || (key0 + q * 16 + row0 <= seen_hi && (n.x | n.y) != 0);
                  *at = make_uint2(v.x & ~n.x, v.y & ~n.y);
                }
              }
              goto again;
            }
          }
          uint32_t ratio[kBatch / C::kChunks];
#pragma unroll
          for (int i = 0; i < kBatch / C::kChunks; ++i) ratio[i] = ratios[b / C::kChunks + i];
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
        mbar_arrive_warp(bar((values ? C::kBarRawVEmpty : C::kBarRawKEmpty) + rs));
      }
      gs0 += pc.steps;
    }
  } else {
    regs_increase<176>();
    // ------------------------------------------------------------ softmax
    const int t = warp / 4;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * kBN;
    const uint32_t tO = tmem + lane_base + C::kColO + t * D;
    uint8_t* q_tile = smem + C::kQOff + t * C::kTileBytes;
    // ring position, and this tile's steps and pieces with steps, before this piece
    int gs0 = 0, done = 0, finals = 0;
    Piece pc;
    bool ok = get_piece(0, &pc);
    // The queries of a piece, fetched while the piece before it is written
    // back: this warp's 32 rows, a row's 16-byte units in consecutive lanes.
    // (Each lane a row of its own would be 32 lines per load: 3 us for the
    // eight warps instead of the latency of one load.)
    constexpr int kUnitsPerRow = D / 8, kRowsPerLoad = 32 / kUnitsPerRow;
    const int q_unit = lane % kUnitsPerRow, q_row = (warp & 3) * 32 + lane / kUnitsPerRow;  // + kRowsPerLoad per load
    uint4 qw[kUnitsPerRow];
    auto fetch_query = [&](const Piece& x) {
      const bool takes_part = !x.end && (t == 0 ? x.b0 > x.a0 : x.b1 > x.a1);
#pragma unroll
      for (int u = 0; u < kUnitsPerRow; ++u) {
        const int r = x.r0 + t * kBM + q_row + u * kRowsPerLoad, i = a.g.div(r);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(x.row0 + i) * a.q_stride +
                                                          (x.h * a.g.G + (r - i * a.g.G)) * D);
        qw[u] = takes_part && r < x.rows ? src[q_unit] : make_uint4(0, 0, 0, 0);
      }
    };
    // Where 16-byte unit u of row tr of the query tile lies.
    auto q_at = [&](int tr, int u) {
      return reinterpret_cast<uint4*>(q_tile + (u >> 3) * C::kChunkBytes + tr * 128 + (((u & 7) ^ (tr & 7)) << 4));
    };
    if (ok) fetch_query(pc);
    for (int np = 0; ok && !pc.end; ++np) {
      const int rows = pc.rows, row0_tile = pc.r0 + t * kBM, h = pc.h, seq = pc.seq;
      const int step0 = t == 0 ? pc.a0 : pc.a1, n_mine = (t == 0 ? pc.b0 : pc.b1) - step0;
      const int r = row0_tile + (threadIdx.x & 127);  // packed row
      const bool live = r < rows;
      const int i = live ? a.g.div(r) : 0, hd = h * a.g.G + (live ? r - i * a.g.G : 0);
      const int p_first = pc.p0 + a.g.div(row0_tile), p_last = pc.p0 + a.g.div(min(row0_tile + kBM, rows) - 1);
      const int p = live ? pc.p0 + i : p_last;
      const int full_lo = pc.full_lo, full_hi = pc.full_hi;
      float qf = 0.f;
      if (n_mine > 0) {
        // scaled into f16 by a power of two (exact within 2^27 of the row's largest value), a thread a row
#pragma unroll
        for (int u = 0; u < kUnitsPerRow; ++u) *q_at(q_row + u * kRowsPerLoad, q_unit) = qw[u];
        __syncwarp();
        const int tr = threadIdx.x & 127;
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < kUnitsPerRow; ++u) {
          qw[u] = *q_at(tr, u);
          const uint32_t x[4] = {qw[u].x, qw[u].y, qw[u].z, qw[u].w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m = max3(m, fabsf(__uint_as_float(x[q] << 16)), fabsf(__uint_as_float(x[q] & 0xffff0000u)));
        }
        int k = 13 - exponent_of(m);
        k = m == 0.f ? 0 : min(max(k, -126), 126);
        const float up = pow2i(k);
        qf = a.scale_log2 * pow2i(-k);
#pragma unroll
        for (int u = 0; u < kUnitsPerRow; ++u) {
          const uint32_t x[4] = {qw[u].x, qw[u].y, qw[u].z, qw[u].w};
          uint32_t f[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            f[q] = pack_f16(__uint_as_float(x[q] << 16) * up, __uint_as_float(x[q] & 0xffff0000u) * up);
          *q_at(tr, u) = make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_async_smem();
        mbar_arrive_warp(bar(C::kBarQFull + t));
      }

      float ms = -INFINITY, mt = -INFINITY, l = 0.f;  // references (log2 units) and denominator
      for (int u = 0; u < n_mine; ++u) {
        const int key0 = pc.key0 + (step0 + u) * kBN;
        ok = mbar_wait_w(bar(C::kBarSFull + t), (done + u) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const TileInfo& ti = infos[(gs0 + step0 + u) % kInfos];
        if (key0 + kBN - 1 > p_first || (a.window > 0 && key0 <= p_last - a.window)) {
          // Some row does not see some key: columns outside [lo, hi) of S
          // become -infinity in tensor memory. A rolled loop of its own: with
          // the selects inside the unrolled code below, that code no longer
          // fits the instruction cache next to the other roles' (2048 queries
          // over 8192 keys, hardly any of whose tiles are cut: 430 us, not 403).
          const int hi = p + 1 - key0, lo = a.window > 0 ? p - a.window + 1 - key0 : 0;
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            const uint32_t bits = low_bits(hi - 32 * w) & ~low_bits(lo - 32 * w);
            uint32_t y[32];
            tmem_ld32(tS + 32 * w, y);
            tmem_ld_wait(y);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1u)) y[c] = 0xff800000u;
            tmem_st32(tS + 32 * w, y);
          }
          tmem_st_wait();
        }
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
        const float sl2 = fmaxf(qf * ti.ek, kLeast), ev = ti.ev;
        const bool by_group = ti.by_group != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
        float x[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c >> 5][c & 31]);
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
              // (no page: no key of the group takes part)
              y[c] = kr >= 0.f ? __uint_as_float(w[c]) * fmaxf(sl2 * kr, kLeast) : -INFINITY;
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
      if (!ok) break;
      Piece nx;
      ok = get_piece(np + 1, &nx);
      if (!ok) break;
      fetch_query(nx);
      // (while the last P.V is computed)
      const float su = ms == -INFINITY ? 0.f : ms, tu = mt == -INFINITY ? 0.f : mt;
      const float f = l == 0.f ? 0.f : ex2(tu - su - kPShift) / l;
      const float lse2 = l == 0.f ? -INFINITY : su + log2f(l);
      if (n_mine > 0) ok = mbar_wait_w(bar(C::kBarOFinal + t), finals & 1, abort_flag);
      if (!ok) break;
      if (n_mine > 0) ++finals;
      done += n_mine;
      gs0 += pc.steps;
      if (row0_tile >= rows) {
        pc = nx;
        continue;
      }
      tc_fence_after();
      const long long at = static_cast<long long>(pc.row0 + i) * a.Hq + hd;
      const long long part = static_cast<long long>(pc.slot) * 2 * kBM + t * kBM;  // the tile's first row there
      if (pc.whole) {
        if (live) a.lse[at] = kLn2 * lse2;
      } else {
        a.part_lse[part + (threadIdx.x & 127)] = lse2;
      }
      if (n_mine == 0) {  // no row of the tile sees a key of the piece
        if (pc.whole && live) {
          uint4* dst = reinterpret_cast<uint4*>(a.o + at * D);
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
        }
        pc = nx;
        continue;
      }
      // As in the forward: 32 rows x 128 bytes at a time through this warp's
      // part of the Q tile (free by now), so that rows leave as whole lines: 64
      // channels of bf16, or 32 of a piece's fp32.
      uint8_t* blk = q_tile + (warp & 3) * 4096;
      uint8_t* mine = blk + lane * 128;
      const int wr = (warp & 3) * 32;  // first row of the warp in the tile
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait(o);
        if (pc.whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = pack_bf16(__uint_as_float(o[8 * e + 2 * q]) * f, __uint_as_float(o[8 * e + 2 * q + 1]) * f);
            *reinterpret_cast<uint4*>(mine + (((4 * (c & 1) + e) ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if ((c & 1) == 0) continue;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(mine + ((e ^ (lane & 7)) * 16)) =
                make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                            __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
        }
        __syncwarp();
#pragma unroll 2  // (code that runs once an item is fetched anew each time: all eight cost 2 to 4 % more)
        for (int j = 0; j < 8; ++j) {
          const int rr = 4 * j + (lane >> 3), v = lane & 7;
          const uint4 val = *reinterpret_cast<const uint4*>(blk + rr * 128 + ((v ^ (rr & 7)) * 16));
          const int pr = row0_tile + wr + rr;
          if (pr < rows) {
            if (pc.whole)
              *reinterpret_cast<uint4*>(a.o + row_at(a, pc.row0, h, pr) * D +
                                        (c >> 1) * 64 + v * 8) = val;
            else
              *reinterpret_cast<uint4*>(a.part_o + (part + wr + rr) * D + c * 32 + v * 4) = val;
          }
        }
        __syncwarp();
      }
      if (*nan_flag && live) {
        // a NaN code was taken out of a tile that not every row sees: put it into the rows that do
        int from = max(pc.key0, first_seen(p, a.window));
        if ((from & ~15) >= full_lo) from = max(from, (full_hi + 1) & ~15);  // nothing is cut before
#pragma unroll 1
        for (int j = from; j <= min(p, pc.key0 + pc.steps * kBN - 1); ++j) {
          const int j0 = j & ~15;
          if (j0 + 15 <= full_hi && j0 >= full_lo) continue;
          const int page = paged_page(a.batch, seq, j >> a.batch.page_shift, a.status);
          if (page < 0) continue;
          const uint8_t* code = a.v_pages + ((static_cast<long long>(page) * a.Hkv + h) * a.batch.page_size +
                                             (j & (a.batch.page_size - 1))) * D;
#pragma unroll 1
          for (int c = 0; c < D; ++c) {
            if ((c & 15) == 0) {  // sixteen codes at a time
              const uint4 w = *reinterpret_cast<const uint4*>(code + c);
              if ((nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w)) == 0) {
                c += 15;
                continue;
              }
            }
            if ((code[c] & 0x7f) != 0x7f) continue;
            if (pc.whole)
              a.o[at * D + c] = __float2bfloat16(__int_as_float(0x7fffffff));
            else
              a.part_o[(part + (threadIdx.x & 127)) * D + c] = __int_as_float(0x7fffffff);
          }
        }
      }
      pc = nx;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(a.status, kStatusTimeout);
}

// Joins the pieces of an item that parts c, c + 1, ... share, by the rule of
// fa_paged_attn.cu's join. Blocks 8 c .. 8 c + 7 take 32 rows each of the item
// that part c begins and does not end, if there is one. Eight threads per row.
template <int D>
__global__ void __launch_bounds__(256) paged_chunk_join_kernel(const ChunkArgs a) {
  constexpr int kCols = D / 8;
  grid_dep_wait();  // (no early launch of the next kernel: see fa_paged.cuh)
  const int c = blockIdx.x / 8;
  const JoinRecord rec = a.records[c];
  if (rec.parts == 0) return;
  const int row = blockIdx.x % 8 * 32 + static_cast<int>(threadIdx.x >> 3), c0 = (threadIdx.x & 7) * kCols;
  const int r = rec.r0 + row;
  if (r >= rec.rows) return;
  float m = -INFINITY, sum = 0.f, x[kCols] = {};
  for (int k = c; k < c + rec.parts; ++k) {
    const long long at = (static_cast<long long>(k) * 2 + (k == c ? 1 : 0)) * 2 * kBM + row;
    const float ls = a.part_lse[at];
    if (ls == -INFINITY) continue;  // (nothing of the row: its channels were not written)
    const float mx = fmaxf(m, ls), alpha = ex2(m - mx), w = ex2(ls - mx);
    sum = fmaf(sum, alpha, w);
    const float* src = a.part_o + at * D + c0;
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(src + i);
      x[i] = fmaf(x[i], alpha, w * v.x);
      x[i + 1] = fmaf(x[i + 1], alpha, w * v.y);
      x[i + 2] = fmaf(x[i + 2], alpha, w * v.z);
      x[i + 3] = fmaf(x[i + 3], alpha, w * v.w);
    }
    m = mx;
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  const long long at = row_at(a, rec.row0, rec.h, r);
  uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + c0);
#pragma unroll
  for (int i = 0; i < kCols; i += 8)
    dst[i / 8] = make_uint4(pack_bf16(x[i] * f, x[i + 1] * f), pack_bf16(x[i + 2] * f, x[i + 3] * f),
                            pack_bf16(x[i + 4] * f, x[i + 5] * f), pack_bf16(x[i + 6] * f, x[i + 7] * f));
  if (c0 == 0) a.lse[at] = sum == 0.f ? -INFINITY : kLn2 * (m + log2f(sum));
}

template <int D>
int launch_chunk_d(const PagedPool& pool, const ChunkArgs& a, int ctas, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap mk, mv;
  const int blocks = pool.num_pages * pool.num_heads;
  if (!make_map_pages(&mk, pool.k_pages, blocks, pool.page_size, D, pool.page_size, false) ||
      !make_map_pages(&mv, pool.v_pages, blocks, pool.page_size, D, pool.page_size, false))
    return -3;
  auto kern = paged_chunk_kernel<D>;
  // attribute slots 28, 29
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, D == 64 ? 28 : 29)) return -3;
  cudaError_t e = launch_overlapped(kern, dim3(ctas), dim3(kThreads), C::kSmemBytes, stream, mk, mv, a);
  if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) return -3;
  e = launch_overlapped(paged_chunk_join_kernel<D>, dim3(8 * (ctas - 1)), dim3(256), 0, stream, a);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace

size_t paged_chunk_workspace_bytes(int d, int ctas) {
  return static_cast<size_t>(ctas) * (2 * 2 * kBM * (d + 1) * sizeof(float) + sizeof(JoinRecord));
}

int launch_paged_chunk(const PagedPool& pool, const PagedBatchDev& batch, const PagedAttn& p, int ctas,
                       void* workspace, cudaStream_t stream) {
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
  a.g = GroupDiv::of(p.Hq / pool.num_heads);
  a.window = p.window;
  // 0 gives uniform weights: S is multiplied by kLeast at least
  a.scale_log2 = p.scale * kLog2e;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + static_cast<size_t>(ctas) * 2 * 2 * kBM * pool.d;
  a.records = reinterpret_cast<JoinRecord*>(a.part_lse + static_cast<size_t>(ctas) * 2 * 2 * kBM);
  return pool.d == 64 ? launch_chunk_d<64>(pool, a, ctas, stream) : launch_chunk_d<128>(pool, a, ctas, stream);
}

}  // namespace fa
