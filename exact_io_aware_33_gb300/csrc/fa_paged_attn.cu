// Attention over a paged e4m3 cache for few query rows (decode, verification
// of drafted tokens): split key ranges, and the merge of their states.
//
// Mathematics. A cached key is kc * sk and a value vc * sv, with codes kc, vc
// and one scale pair per page and head, so with S = scale q . kc sk the output
// row is sum_j 2^(s_j) sv_j vc_j / sum_j 2^(s_j), s = S log2 e. The numerator
// is carried relative to its own maximum m_t = max_j (s_j + log2 sv_j) and the
// denominator relative to m_s = max_j s_j: the weights P_j = 2^(s_j + log2
// sv_j - m_t) then lie in (0, 1] whatever the scales, the codes enter the
// tensor core as they are (an e4m3 value is exact in f16), and no cached
// element is ever multiplied by its scale. All statistics and sums are fp32.
//
// Precision. Queries are scaled per row by a power of two into f16's normal
// range (exact for every bf16 value within 2^27 of the row's largest; below
// that it would change S by less than 2^-38 of its bound). P is rounded to f16
// (2^-12 of it) after a factor of 2^6, so that weights down to 2^-20 of their
// reference keep that precision and those down to 2^-31 still count; the
// references lie between the largest weight so far and 2^-8 of it (as in the
// forward). The denominator adds the weights before that rounding.
//
// What bounds it: at one token per sequence every cached byte is read once
// for G = Hq / Hkv rows of arithmetic, far below the tensor core's rate, so
// the kernel is a copy from HBM. It therefore is organised as one: a TMA warp
// keeps a ring of tiles (64 keys, or 128 at d = 64) full and four warps take a
// quarter of each tile, each with an online softmax of its own, so that no two
// warps wait for one another until the end of an item. Codes go from shared
// memory to registers and are widened there (mma.sync takes its operands from
// registers; tcgen05 would want them widened in shared memory first, which
// costs a second pass over it).
//
// Division of the work. An item is one sequence, key head and tile of 8 or 16
// query rows. The streaming form cuts the tiles of all items, laid end to end, into
// equal parts, one per CTA slot of the GPU: lengths differ by orders of
// magnitude between the sequences of a batch, and a part may hold many short
// items or a piece of a long one. The ring runs on across items. Items that
// end up in one part are written at once; pieces go to the workspace (two per
// part at most: one that it continues and one that it leaves) and a second
// kernel joins them. Where the whole batch is so little that a second launch
// would cost more than it divides, a cluster of CTAs takes an item instead
// and joins its pieces through distributed shared memory.

#include <cmath>

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kGroup = 16;       // keys of one mma tile; a page is one or more groups
constexpr int kThreads = 160;    // four warps and the TMA warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 6.f;   // P is held as 2^6 P
constexpr float kSlack = 8.f;    // log2 units that a weight may pass its reference by

// Each item costs about this many tiles more than it has (its queries, the
// joining of its four warps, the write-back).
constexpr int kItemUnits = 2;
constexpr int kPartUnits = 4;  // a part has at least this many units, and so a tile of an item that it continues

// Keys per stage. At d = 64 a tile of 64 would be 8 KiB for the same waiting,
// voting and reference keeping, and those, not the bytes, would set the pace.
template <int D>
constexpr int kTileOf = D == 64 ? 128 : 64;

// NB: blocks of eight query rows per CTA.
template <int D, int NB>
struct Cfg {
  static constexpr int kTile = kTileOf<D>;
  static constexpr int kGpt = kTile / kGroup;  // groups per tile
  static constexpr int kGpw = kGpt / 4;        // and per warp
  static constexpr int kRows = 8 * NB;
  static constexpr int kCtasPerSm = NB == 1 ? 3 : 2;
  static constexpr int kTileBytes = kTile * D;
  // the four warps' states at the end of an item: rows of d channels, then {m_s, m_t, l, -} each
  static constexpr int kPitch = D + 4;
  static constexpr int kStateBytes = 4 * kRows * (kPitch + 4) * 4;
  // as many stages as leave room for the other CTAs of the SM
  static constexpr int kRoom = 233472 / kCtasPerSm - 1024 - 1024 - 768 - kStateBytes;
  static constexpr int kStages = kRoom / (2 * kTileBytes) < 10 ? kRoom / (2 * kTileBytes) : 10;
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kStages * kTileBytes;
  static constexpr int kStateOff = 2 * kStages * kTileBytes;
  static constexpr int kScaleOff = kStateOff + kStateBytes;  // [stage][group] {sk, log2 sv}
  static constexpr int kBarOff = kScaleOff + kStages * kGpt * 8;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;  // + slack to align the base
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "the CTAs of an SM must fit");
};

struct AttnArgs {
  PagedBatchDev batch;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [part][2][16][d], normalised
  float* part_lse;  // [part][2][16], log2 units
  JoinRecord* records;  // [part]
  const uint8_t* v_pages;  // the rare path that looks for NaN codes again
  const float* k_scales;
  const float* v_scales;
  int* status;
  int Hq, Hkv;
  GroupDiv g;  // G = Hq / Hkv
  int window;
  int row_tiles;   // cluster form: row tiles of the longest packed sequence
  int cluster;     // CTAs per item (cluster form)
  float scale_log2;
};

// Where row r of a key head stands in o and lse: (token, query head).
__device__ __forceinline__ long long row_at(const AttnArgs& a, int row0, int h, int r) {
  const int i = a.g.div(r);
  return static_cast<long long>(row0 + i) * a.Hq + h * a.g.G + (r - i * a.g.G);
}

// One sequence's items: its tiles of R rows, and the tiles of kTile keys that any
// of its queries sees.
struct SeqGeo {
  PagedSeq s;
  int rows, rts;  // packed (query, head of the group) rows of a key head, and tiles of R of them
  int p0;         // position of query 0
  int t0, nt;
};

template <int R, int kTile>
__device__ __forceinline__ SeqGeo seq_geo(const AttnArgs& a, int seq) {
  SeqGeo g;
  g.s = paged_seq(a.batch, seq, a.status);
  g.rows = g.s.n * a.g.G;
  g.rts = (g.rows + R - 1) / R;
  g.p0 = g.s.len - g.s.n;
  const int hi = g.s.n > 0 ? g.s.len : 0;
  const int lo = first_seen(g.p0, a.window);
  g.t0 = lo / kTile;
  g.nt = hi > lo ? (hi + kTile - 1) / kTile - g.t0 : 0;
  return g;
}

__device__ __forceinline__ long long seq_units(const AttnArgs& a, const SeqGeo& g) {
  return static_cast<long long>(a.Hkv) * g.rts * (g.nt + kItemUnits);
}

// The rows of an item and the keys [lo, hi) that any of them sees.
struct RowTile {
  int rows, r0;
  int p0;
  int p_lo, p_hi;  // positions of the first and last query of the tile
  int lo, hi;
};

template <int R>
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, const SeqGeo& s, int rt) {
  RowTile g;
  g.rows = s.rows;
  g.r0 = rt * R;
  g.p0 = s.p0;
  g.p_lo = g.p0 + a.g.div(g.r0);
  g.p_hi = g.p0 + a.g.div(min(g.r0 + R, g.rows) - 1);
  g.hi = max(g.p_hi + 1, 0);
  g.lo = first_seen(g.p_lo, a.window);
  return g;
}

// x / y for x >= 0, y > 0: by 32 bits where they suffice, which takes a fifth of the time.
__device__ __forceinline__ long long div_pos(long long x, int y) {
  if (x >> 32) return x / y;
  return static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}
__device__ __forceinline__ void split_by(long long x, int y, int* quotient, int* remainder) {
  const long long q = div_pos(x, y);
  *quotient = static_cast<int>(q);
  *remainder = static_cast<int>(x - q * y);
}

// First unit of part c of `parts` over `units` units, and the part of a unit.
__device__ __forceinline__ long long part_start(long long units, int parts, int c) {
  return div_pos(units * c, parts);
}

// The units of the sequences, by one warp: their total, and, kept from that
// pass, the first 32 sequences' (what a batch of up to 32 needs no second
// pass over the lengths for).
template <int R, int kTile>
struct Units {
  long long total;
  long long own, end;  // of sequence lane_id(): its units, and the units up to its end

  __device__ __forceinline__ void scan(const AttnArgs& a, int b0, long long before) {
    const int b = b0 + static_cast<int>(lane_id());
    own = b < a.batch.B ? seq_units(a, seq_geo<R, kTile>(a, b)) : 0;
    end = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, end, m);
      if (lane_id() >= static_cast<uint32_t>(m)) end += x;
    }
    end += before;
  }
  __device__ __forceinline__ void start(const AttnArgs& a) {
    scan(a, 0, 0);
    total = __shfl_sync(0xffffffffu, end, 31);
    if (a.batch.B > 32) {
      long long sum = 0;
      for (int b = 32 + static_cast<int>(lane_id()); b < a.batch.B; b += 32) sum += seq_units(a, seq_geo<R, kTile>(a, b));
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      total += sum;
    }
  }
  // The sequence that holds unit u (below the total), and its first unit.
  __device__ __forceinline__ int find(const AttnArgs& a, long long u, long long* first) {
    for (int b0 = 0; b0 < a.batch.B; b0 += 32) {
      if (b0 > 0) scan(a, b0, __shfl_sync(0xffffffffu, end, 31));
      const uint32_t past = __ballot_sync(0xffffffffu, end > u);
      if (past) {
        const int i = __ffs(past) - 1;
        *first = __shfl_sync(0xffffffffu, end - own, i);
        return b0 + i;
      }
    }
    *first = 0;  // not reached for u below the total
    return a.batch.B;
  }
};

// Walks the pieces of items that a CTA has, sequence by sequence: tiles
// [v0, v1) of the sequence's tiles laid end to end, item after item (key head
// by key head, row tile by row tile). A sequence whose rows see no key has
// items [e0, e1) to be filled with zeros instead. Every warp walks alike.
template <int R, int kTile>
struct Walk {
  long long u0, u1;  // this CTA's units
  long long units;   // of the whole batch, in `parts` parts
  int parts;
  long long base;    // first unit of sequence b
  long long seq0;    // and of the sequence that next() gave
  int b;

  __device__ __forceinline__ void start(const AttnArgs& a, int part, int ctas) {
    Units<R, kTile> all;
    all.start(a);
    units = all.total;
    parts = static_cast<int>(min(static_cast<long long>(ctas), max(units / kPartUnits, 1LL)));
    u0 = part_start(units, parts, min(part, parts));
    u1 = part_start(units, parts, min(part + 1, parts));
    b = a.batch.B;
    base = 0;
    if (u0 < u1) b = all.find(a, u0, &base);
  }
  // unit -> tile index in the sequence: the first kItemUnits of an item are not tiles
  static __device__ __forceinline__ long long tile_of(long long u, int nt) {
    int item, rest;
    split_by(u, nt + kItemUnits, &item, &rest);
    return static_cast<long long>(item) * nt + max(rest - kItemUnits, 0);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, SeqGeo* g, long long* v0, long long* v1, int* e0,
                                       int* e1) {
    while (b < a.batch.B && base < u1) {
      *g = seq_geo<R, kTile>(a, b);
      const long long own = seq_units(a, *g);
      const long long lo = max(u0 - base, 0LL), hi = min(u1 - base, own);
      seq0 = base;
      base += own;
      ++b;
      if (hi <= lo) continue;
      *v0 = *v1 = 0;
      *e0 = *e1 = 0;
      if (g->nt > 0) {
        *v0 = tile_of(lo, g->nt);
        *v1 = tile_of(hi, g->nt);
        if (*v1 > *v0) return true;
      } else {
        *e0 = static_cast<int>((lo + kItemUnits - 1) / kItemUnits);
        *e1 = static_cast<int>((hi + kItemUnits - 1) / kItemUnits);
        if (*e1 > *e0) return true;
      }
    }
    return false;
  }
};

// Whether every row of the tile sees every one of the 16 keys from j0 on.
__device__ __forceinline__ bool all_see(const RowTile& g, int j0, int window) {
  return j0 + kGroup - 1 <= g.p_lo && (window == 0 || j0 > g.p_hi - window);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 block of 16-bit values, in the fragment layout of mma.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// Over the eight lanes of equal lane & 3.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// One row's D/4 consecutive queries of this lane, scaled into f16, and the
// factor that undoes it (with the softmax scale). Four words of eight values
// per 16 bytes; word pairs are the two halves of an mma step's k range.
template <int D>
__device__ __forceinline__ float load_query(const __nv_bfloat16* row, bool on, float scale_log2,
                                            uint32_t (&w)[D / 8]) {
  uint4 raw[D / 32];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    raw[i] = on ? *reinterpret_cast<const uint4*>(row + 8 * i) : make_uint4(0, 0, 0, 0);
    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = max3(m, fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xffff0000u)));
  }
  m = quad_max(m);
  // largest of the row into [2^13, 2^14)
  int k = 13 - (static_cast<int>(__float_as_uint(m) >> 23) - 127);
  k = m == 0.f ? 0 : min(max(k, -126), 126);
  const float up = pow2i(k);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[4 * i + j] = pack_f16(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xffff0000u) * up);
  }
  return scale_log2 * pow2i(-k);
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// kCols channels from c0 on of row r of a key head.
template <int D, int kCols>
__device__ __forceinline__ void store_row(const AttnArgs& a, const SeqGeo& sg, int h, int r, int c0,
                                          const float (&x)[kCols], float lse2) {
  const long long at = row_at(a, sg.s.row0, h, r);
  __nv_bfloat16* dst = a.o + at * D + c0;
#pragma unroll
  for (int i = 0; i < kCols; i += 4)
    *reinterpret_cast<uint2*>(dst + i) = make_uint2(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]));
  if (c0 == 0) a.lse[at] = kLn2 * lse2;
}

// kCluster: the cluster form (see the top of the file).
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys (and
// channels) fill the 16 rows of an mma tile and queries its 8 columns, so that
// eight query rows, the usual group, leave nothing idle, and a widened key or
// value serves all NB blocks of them. P^T comes out of the softmax as the
// transpose of what the second product takes, two 8 x 8 blocks per 16 keys.
template <int D, int NB, bool kCluster>
__global__ void __launch_bounds__(kThreads, Cfg<D, NB>::kCtasPerSm)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const AttnArgs a) {
  using C = Cfg<D, NB>;
  constexpr int kS = C::kStages, R = C::kRows, kTile = C::kTile, kGpt = C::kGpt, kGpw = C::kGpw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const uint32_t full = sb + C::kBarOff, empty = full + 8 * kS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* nan_flag = abort_flag + 1;  // two, taken in turn by the items
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 4);
    }
    *abort_flag = 0;
    nan_flag[0] = nan_flag[1] = 0;
    mbar_fence_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();

  // What this CTA does: a walk over its part (streaming), or its piece of one
  // item (cluster; `rank` of `pieces` that have any tile).
  Walk<R, kTile> walk;
  SeqGeo sg;
  long long v0 = 0, v1 = 0;
  int e0 = 0, e1 = 0, rank = 0, pieces = 1;
  bool more;
  if constexpr (kCluster) {
    rank = static_cast<int>(blockIdx.x % a.cluster);
    const long long item = blockIdx.x / a.cluster;
    const int rt = static_cast<int>(item % a.row_tiles);
    const long long bh = item / a.row_tiles;
    const int h = static_cast<int>(bh % a.Hkv);
    sg = seq_geo<R, kTile>(a, static_cast<int>(bh / a.Hkv));
    if (rt >= sg.rts) return;  // the whole cluster alike
    walk.b = static_cast<int>(bh / a.Hkv) + 1;
    const int own = h * sg.rts + rt;
    const int per = (sg.nt + a.cluster - 1) / a.cluster;
    pieces = sg.nt > 0 ? (sg.nt + per - 1) / per : 1;
    if (rank >= pieces) return;  // nothing to do, and nothing that the others would read
    v0 = static_cast<long long>(own) * sg.nt + min(rank * per, sg.nt);
    v1 = static_cast<long long>(own) * sg.nt + min((rank + 1) * per, sg.nt);
    if (sg.nt == 0) {
      e0 = own;
      e1 = own + 1;
    }
    more = true;
  } else {
    walk.start(a, blockIdx.x, gridDim.x);
    more = walk.next(a, &sg, &v0, &v1, &e0, &e1);
  }
  uint32_t it = 0;  // tiles so far: the ring runs on across items and sequences

  if (warp == 4) {
    // ------------------------------------------------------------ TMA warp
    // Lane i looks up the i-th of 32 groups of 16 keys (four or eight tiles,
    // across items of a sequence): its page, then its scales. The next tiles'
    // two dependent loads are under way while the present ones are issued. The
    // lane of a box's first group issues its copies.
    constexpr int kBatch = 32 / kGpt;  // tiles looked up at once
    const int tile_in = lane / kGpt, grp = lane % kGpt;
    const int box_rows = min(a.batch.page_size, kTile), per_box = box_rows / kGroup;
    const uint32_t box_bytes = 2u * box_rows * D;  // of K and V
    JoinRecord record{};
    // Whether to go on: the verdict of the whole warp, so that its lanes leave
    // the loops together. (The flag itself may be raised between two lanes' reads.)
    bool ok = true;
    while (more && ok) {
      const int seq = walk.b - 1;
      if (!kCluster && sg.nt > 0) {
        int item, end;  // of the last tile here
        split_by(v1 - 1, sg.nt, &item, &end);
        if (end + 1 < sg.nt && v0 <= static_cast<long long>(item) * sg.nt) {  // begun and not ended
          const int h = item / sg.rts;
          record = JoinRecord{parts_until(walk.seq0 + (item + 1LL) * (sg.nt + kItemUnits), walk.units, walk.parts, blockIdx.x),
                              sg.s.row0, h, (item - h * sg.rts) * R, sg.rows, {}};
        }
      }
      long long left = v1 - v0;  // tiles not looked up yet
      int item = 0, tile = 0;
      if (sg.nt > 0) split_by(v0, sg.nt, &item, &tile);
      int n_page = -1, n_head = 0, n_key = 0, n_count = 0;
      auto look = [&]() {  // the next (up to) kBatch tiles' pages
        n_count = static_cast<int>(min(left, static_cast<long long>(kBatch)));
        int ti = tile + tile_in, ii = item;
        while (ti >= sg.nt && sg.nt > 0) {
          ti -= sg.nt;
          ++ii;
        }
        n_page = -1;
        if (tile_in < n_count) {
          n_head = sg.rts == 1 ? ii : ii / sg.rts;
          const RowTile g = row_tile<R>(a, sg, ii - n_head * sg.rts);
          n_key = (sg.t0 + ti) * kTile + grp * kGroup;
          if (n_key < g.hi && n_key + kGroup > g.lo)
            n_page = paged_page(a.batch, seq, n_key >> a.batch.page_shift, a.status);
        }
        left -= n_count;
        tile += n_count;
        while (tile >= sg.nt && sg.nt > 0) {
          tile -= sg.nt;
          ++item;
        }
      };
      float n_sk = -1.f, n_sv = 1.f;
      auto scales = [&]() {
        n_sk = -1.f;
        if (n_page >= 0) {
          const long long at = static_cast<long long>(n_page) * a.Hkv + n_head;
          n_sk = a.k_scales[at];
          n_sv = a.v_scales[at];
        }
      };
      look();
      scales();
      while (n_count > 0 && ok) {
        int box_page = n_page;  // of this lane's box: its groups share a page, or have none to read
        const int head = n_head, key = n_key, count = n_count;
        const float sk = n_sk, sv = n_sv;
        look();
        if (per_box > 1) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 1));
        if (per_box > 2) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 2));
        if (per_box > 4) box_page = max(box_page, __shfl_xor_sync(0xffffffffu, box_page, 4));
        const bool issues = grp % per_box == 0 && box_page >= 0;
        const uint32_t issuers = __ballot_sync(0xffffffffu, issues);
        const int slot = key & (a.batch.page_size - 1), blk = box_page * a.Hkv + head;
        const uint32_t off = grp * kGroup * D;
        for (int i = 0; i < count; ++i) {
          const int st = it % kS;
#ifdef FA_TEST_SKIP_ARRIVE
          // Test-only build (never in libfa.so): a sequence's last tile is
          // never loaded, so the four warps' bounded waits for it run out and
          // the CTA winds down through the abort path.
          if (n_count == 0 && i == count - 1) break;
#endif
          if (it >= kS) ok = mbar_wait_w(empty + 8 * st, (it / kS - 1) & 1, abort_flag);
          if (!ok) break;
          if (tile_in == i) {
            // the copies need the pages only: they go out before the scales are waited for
            if (issues) {
              tma_load_3d(sb + C::kKOff + st * C::kTileBytes + off, &tmK, full + 8 * st, 0, slot, blk);
              tma_load_3d(sb + C::kVOff + st * C::kTileBytes + off, &tmV, full + 8 * st, 0, slot, blk);
            }
            const uint32_t bits = __float_as_uint(sv);
            // exact for the powers of two that the append writes
            const float ev = (bits & 0x7fffffu) ? log2f(sv)
                             : bits == 0       ? -INFINITY
                                               : static_cast<float>(static_cast<int>(bits >> 23) - 127);
            *reinterpret_cast<float2*>(smem + C::kScaleOff + (st * kGpt + grp) * 8) = make_float2(sk, ev);
          }
          __syncwarp();
          // (bytes that have landed already count as well: the phase cannot end before this arrival)
          if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, __popc(issuers & (((1u << kGpt) - 1) << (kGpt * i))) * box_bytes);
          if (i == min(kBatch / 2 - 1, count - 1)) scales();
          ++it;
        }
        __syncwarp();
      }
      if (ok) more = kCluster ? false : walk.next(a, &sg, &v0, &v1, &e0, &e1);
    }
    if (!kCluster && lane == 0) a.records[blockIdx.x] = record;
    // let every copy in flight land before the CTA can end
    for (uint32_t i = it > kS ? it - kS : 0; i < it; ++i) mbar_wait(full + 8 * (i % kS), (i / kS) & 1, nullptr);
    if (lane == 0 && *abort_flag) atomicExch(a.status, kStatusTimeout);
    if constexpr (kCluster) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- four compute warps
  const int n = lane >> 2, t = lane & 3;  // fragment row (or column) and quarter
  constexpr int kTpr = 128 / R;           // at the end of an item: threads per row,
  constexpr int kCols = D / kTpr;         // and channels per thread
  const int wrow = threadIdx.x / kTpr, c0 = threadIdx.x % kTpr * kCols;
  float* so = reinterpret_cast<float*>(smem + C::kStateOff);  // [warp][row][kPitch]
  float* sst = so + 4 * R * C::kPitch;                        // [warp][row][4]: m_s, m_t, l
  bool ok = true;
  int turn = 0;

  while (more) {
    const int seq = walk.b - 1;
    // items whose rows see no key
    for (int e = e0; e < e1; ++e) {
      const int r = e % sg.rts * R + wrow;
      const float x[kCols] = {};
      if (r < sg.rows) store_row<D>(a, sg, e / sg.rts, r, c0, x, -INFINITY);
    }
    int item = 0, tile = 0;
    if (sg.nt > 0) split_by(v0, sg.nt, &item, &tile);
    for (long long left = v1 - v0; left > 0;) {
      // the piece [tile, tile_end) of this item
      const int tile_end = static_cast<int>(min(static_cast<long long>(sg.nt), tile + left));
      const int h = sg.rts == 1 ? item : item / sg.rts;
      const RowTile g = row_tile<R>(a, sg, item - h * sg.rts);
      uint32_t qb[NB][D / 8];   // B operand of S^T: row n of each block, D/4 channels
      float qf[NB][2];          // per column of the accumulators (rows 2t, 2t + 1 of a block)
      int p_row[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int row = g.r0 + nb * 8 + n;
        const bool on = row < g.rows;
        const int i = on ? a.g.div(row) : 0, hd = h * a.g.G + (on ? row - i * a.g.G : 0);
        const float f = load_query<D>(
            a.q + static_cast<long long>(sg.s.row0 + i) * a.q_stride + hd * D + t * (D / 4), on, a.scale_log2, qb[nb]);
        const int p = on ? g.p0 + i : g.p_hi;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qf[nb][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
          p_row[nb][e] = __shfl_sync(0xffffffffu, p, 4 * (2 * t + e));
        }
      }
      float o[NB][D / 16][4];
      float ms[NB][2], mt[NB][2], l[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
        ms[nb][0] = ms[nb][1] = mt[nb][0] = mt[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
      }
      bool saw_nan = false;

      for (int ti = tile; ti < tile_end; ++ti, ++it) {
        const int st = it % kS;
        ok = ok && mbar_wait_w(full + 8 * st, (it / kS) & 1, abort_flag);
        if (!ok) continue;
        // this warp's groups of 16 keys
        float2 sc[kGpw];
        bool any = false;
#pragma unroll
        for (int q = 0; q < kGpw; ++q) {
          sc[q] = *reinterpret_cast<const float2*>(smem + C::kScaleOff + (st * kGpt + warp * kGpw + q) * 8);
          any = any || !(sc[q].x < 0.f);  // below zero: no row sees these keys, or they have no page
        }
        if (any) {
          const int j0 = (sg.t0 + ti) * kTile + warp * kGpw * kGroup;
          bool part = false;
#pragma unroll
          for (int q = 0; q < kGpw; ++q) part = part || !all_see(g, j0 + q * kGroup, a.window) || sc[q].x < 0.f;
          const uint8_t* kb = smem + C::kKOff + st * C::kTileBytes + warp * kGpw * kGroup * D;
          const uint8_t* vb = smem + C::kVOff + st * C::kTileBytes + warp * kGpw * kGroup * D;
          // S^T = K Q^T: 16 keys x 8 NB rows. A lane holds D/4 consecutive
          // channels of keys n and n + 8, four per mma step, in the order
          // that its queries have. (kb lies on a multiple of eight rows, so a
          // row's swizzle is that of its number here.)
          constexpr int kChains = NB * kGpw == 1 ? 2 : 1;  // of dependent products, where there is only one
          float acc[kGpw][NB][kChains][4] = {};
#pragma unroll
          for (int q = 0; q < kGpw; ++q) {
            uint4 kw[2][D / 64];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int row = q * kGroup + hh * 8 + n;
              if constexpr (D == 128) {
                kw[hh][0] = *reinterpret_cast<const uint4*>(kb + row * 128 + (((2 * t) ^ (row & 7)) << 4));
                kw[hh][1] = *reinterpret_cast<const uint4*>(kb + row * 128 + (((2 * t + 1) ^ (row & 7)) << 4));
              } else {
                kw[hh][0] = *reinterpret_cast<const uint4*>(kb + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
              }
            }
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t ka[4];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const uint32_t w = e == 0 ? kw[hh][c].x : e == 1 ? kw[hh][c].y : e == 2 ? kw[hh][c].z : kw[hh][c].w;
                  ka[hh] = e4m3x2_to_f16x2(static_cast<uint16_t>(w));
                  ka[2 + hh] = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816(acc[q][nb][e % kChains], ka, qb[nb][2 * (4 * c + e)], qb[nb][2 * (4 * c + e) + 1]);
              }
            }
          }
          // x[q][nb][2 hh + e]: key n + 8 hh of group q, row 2t + e, in log2 units
          float x[kGpw][NB][4];
          bool over = false;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int q = 0; q < kGpw; ++q) {
                const float f = qf[nb][e] * sc[q].x;
                const float bar = fminf(ms[nb][e], mt[nb][e] - sc[q].y) + kSlack;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  float v = acc[q][nb][0][2 * hh + e];
                  if constexpr (kChains == 2) v += acc[q][nb][1][2 * hh + e];
                  v *= f;
                  if (part && (sc[q].x < 0.f || !sees(p_row[nb][e], j0 + q * kGroup + n + 8 * hh, a.window)))
                    v = -INFINITY;
                  x[q][nb][2 * hh + e] = v;
                  over = over || v > bar;
                }
              }
            }
          }
          // The references only move when a weight would pass them by more
          // than 2^8; until then weights above 1 are summed as they are.
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float alpha[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float ms_new = ms[nb][e], mt_new = mt[nb][e];
#pragma unroll
                for (int q = 0; q < kGpw; ++q) {
                  const float mx = column_max(fmaxf(x[q][nb][e], x[q][nb][2 + e]));
                  ms_new = fmaxf(ms_new, mx);
                  mt_new = fmaxf(mt_new, mx + sc[q].y);
                }
                // a row that has seen nothing yet has both at -infinity
                l[nb][e] *= ex2(ms[nb][e] - (ms_new == -INFINITY ? 0.f : ms_new));
                alpha[e] = ex2(mt[nb][e] - (mt_new == -INFINITY ? 0.f : mt_new));
                ms[nb][e] = ms_new;
                mt[nb][e] = mt_new;
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[nb][i][0] *= alpha[0];
                o[nb][i][1] *= alpha[1];
                o[nb][i][2] *= alpha[0];
                o[nb][i][3] *= alpha[1];
              }
            }
          }
          uint32_t pb[kGpw][NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float w[kGpw][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float su = ms[nb][e] == -INFINITY ? 0.f : ms[nb][e];
              const float tu = mt[nb][e] == -INFINITY ? 0.f : mt[nb][e];
#pragma unroll
              for (int q = 0; q < kGpw; ++q) {
                const float f2 = ex2(fminf(su + sc[q].y - tu + kPShift, 126.f));
                const float p0 = ex2(x[q][nb][e] - su), p1 = ex2(x[q][nb][2 + e] - su);
                l[nb][e] += p0 + p1;
                w[q][e] = p0 * f2;
                w[q][2 + e] = p1 * f2;
              }
            }
#pragma unroll
            for (int q = 0; q < kGpw; ++q) {
              pb[q][nb][0] = transpose8x8(pack_f16(w[q][0], w[q][1]));
              pb[q][nb][1] = transpose8x8(pack_f16(w[q][2], w[q][3]));
            }
          }
          // O^T += V^T P^T: lane (n, t) takes channels [n D/8, (n + 1) D/8) of
          // keys 2t, 2t+1, 2t+8, 2t+9; an mma tile's rows n and n + 8 are two
          // neighbouring channels
#pragma unroll
          for (int q = 0; q < kGpw; ++q) {
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = q * kGroup + 2 * t + (e & 1) + 8 * (e >> 1);
              if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(vb + row * 128 + ((n ^ (row & 7)) << 4));
                vw[e][0] = w.x; vw[e][1] = w.y; vw[e][2] = w.z; vw[e][3] = w.w;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(
                    vb + row * 64 + (((n >> 1) ^ ((row >> 1) & 3)) << 4) + ((n & 1) << 3));
                vw[e][0] = w.x; vw[e][1] = w.y;
              }
            }
            const bool absent = sc[q].x < 0.f;  // (nothing was loaded)
            if (part && (absent || !all_see(g, j0 + q * kGroup, a.window))) {
              // keys that a row does not see have weight 0, and 0 x NaN is NaN: here
              // NaN codes are taken out, and rows that do see one are mended at the end.
              // (Not for codes behind the last key that any row sees: slots past a
              // length may hold anything, and often do.)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                  const uint32_t z = nan_bytes(vw[e][i]);
                  saw_nan = saw_nan || (z != 0 && !absent && j0 + q * kGroup + 2 * t + (e & 1) + 8 * (e >> 1) <= g.p_hi);
                  vw[e][i] = absent ? 0u : vw[e][i] & ~z;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              // byte pairs of two neighbouring keys, channel by channel
              const uint32_t a01 = __byte_perm(vw[0][i], vw[1][i], 0x5140), a23 = __byte_perm(vw[0][i], vw[1][i], 0x7362);
              const uint32_t b01 = __byte_perm(vw[2][i], vw[3][i], 0x5140), b23 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
              const uint32_t va[2][4] = {
                  {e4m3x2_to_f16x2(static_cast<uint16_t>(a01)), e4m3x2_to_f16x2(static_cast<uint16_t>(a01 >> 16)),
                   e4m3x2_to_f16x2(static_cast<uint16_t>(b01)), e4m3x2_to_f16x2(static_cast<uint16_t>(b01 >> 16))},
                  {e4m3x2_to_f16x2(static_cast<uint16_t>(a23)), e4m3x2_to_f16x2(static_cast<uint16_t>(a23 >> 16)),
                   e4m3x2_to_f16x2(static_cast<uint16_t>(b23)), e4m3x2_to_f16x2(static_cast<uint16_t>(b23 >> 16))}};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma16816(o[nb][2 * i], va[0], pb[q][nb][0], pb[q][nb][1]);
                mma16816(o[nb][2 * i + 1], va[1], pb[q][nb][0], pb[q][nb][1]);
              }
            }
          }
        }
        mbar_arrive_warp(empty + 8 * st);
      }
      if (saw_nan) nan_flag[turn] = 1;

      // ---------------------------------------------------------- join the four warps
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = nb * 8 + 2 * t + e;
          const float sum = column_sum(l[nb][e]);
          float* dst = so + (warp * R + row) * C::kPitch + n * (D / 8);
          // o[nb][i][2 c + e] is channel n D/8 + 2 i + c of row 2t + e
#pragma unroll
          for (int i = 0; i < D / 16; i += 2)
            *reinterpret_cast<float4*>(dst + 2 * i) =
                make_float4(o[nb][i][e], o[nb][i][2 + e], o[nb][i + 1][e], o[nb][i + 1][2 + e]);
          if (n == 0) {
            float* s4 = sst + (warp * R + row) * 4;
            s4[0] = ms[nb][e];
            s4[1] = mt[nb][e];
            s4[2] = sum;
          }
        }
      }
      named_bar_sync(1, 128);
      // a wait that ran out: no results, but every warp goes through the same barriers
      const bool dead = *abort_flag != 0;
      const bool whole = tile == 0 && tile_end == sg.nt;
      float x[kCols] = {}, sum = 0.f, m = -INFINITY;
      if (!dead && g.r0 + wrow < g.rows) {
        float mv = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          m = fmaxf(m, sst[(w * R + wrow) * 4]);
          mv = fmaxf(mv, sst[(w * R + wrow) * 4 + 1]);
        }
        const float mu = m == -INFINITY ? 0.f : m, vu = mv == -INFINITY ? 0.f : mv;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float* s4 = sst + (w * R + wrow) * 4;
          sum += s4[2] * ex2(s4[0] - mu);
          const float f = ex2(s4[1] - vu);
          const float* src = so + (w * R + wrow) * C::kPitch + c0;
#pragma unroll
          for (int i = 0; i < kCols; ++i) x[i] = fmaf(src[i], f, x[i]);
        }
        // sum = 0: the row saw no key
        const float f = sum == 0.f ? 0.f : ex2(vu - mu - kPShift) / sum;
#pragma unroll
        for (int i = 0; i < kCols; ++i) x[i] *= f;
        if (nan_flag[turn]) {
          const int p = g.p0 + a.g.div(g.r0 + wrow);
          for (int j = max((sg.t0 + tile) * kTile, g.lo); j < min((sg.t0 + tile_end) * kTile, g.hi); ++j) {
            if (all_see(g, j & ~(kGroup - 1), a.window)) {
              // on to the first group that the causal edge cuts
              j = max(j | (kGroup - 1), ((g.p_lo + 1) & ~(kGroup - 1)) - 1);
              continue;
            }
            if (!sees(p, j, a.window)) continue;
            const int page = paged_page(a.batch, seq, j >> a.batch.page_shift, a.status);
            if (page < 0) continue;
            const uint8_t* code = a.v_pages +
                                  ((static_cast<long long>(page) * a.Hkv + h) * a.batch.page_size +
                                   (j & (a.batch.page_size - 1))) * D + c0;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if ((code[i] & 0x7f) == 0x7f) x[i] = __int_as_float(0x7fffffff);
          }
        }
        const float lse2 = sum == 0.f ? -INFINITY : m + log2f(sum);
        if (kCluster ? pieces == 1 : whole) {
          store_row<D>(a, sg, h, g.r0 + wrow, c0, x, lse2);
        } else if constexpr (kCluster) {
          // this thread alone read warp 0's part of these channels: the piece's state takes its place
          float* dst = so + wrow * C::kPitch + c0;
#pragma unroll
          for (int i = 0; i < kCols; ++i) dst[i] = x[i];
        } else {
          // piece 0 of the part continues an item, piece 1 begins one
          const long long at = (static_cast<long long>(blockIdx.x) * 2 + (tile == 0 ? 1 : 0)) * R + wrow;
          float* dst = a.part_o + at * D + c0;
#pragma unroll
          for (int i = 0; i < kCols; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          if (c0 == 0) a.part_lse[at] = lse2;
        }
        m = lse2;
      }
      named_bar_sync(1, 128);  // the states have been read
      if (threadIdx.x == 0) nan_flag[turn] = 0;  // next raised two items on, past two more barriers
      turn ^= 1;
      if constexpr (kCluster) {
        if (c0 == 0) sst[wrow * 4] = dead ? -INFINITY : m;
      }
      left -= tile_end - tile;
      tile = 0;
      ++item;
    }
    more = kCluster ? false : walk.next(a, &sg, &v0, &v1, &e0, &e1);
  }
  if (*abort_flag && threadIdx.x == 0) atomicExch(a.status, kStatusTimeout);
  if constexpr (kCluster) {
    // Join the pieces: every CTA of the cluster takes a share of the rows.
    cluster_sync();
    if (pieces > 1 && v1 > v0) {
      const int own = static_cast<int>(v0 / sg.nt);
      const int r = own % sg.rts * R + wrow;
      if (wrow % pieces == rank && r < sg.rows && !*abort_flag) {
        float m = -INFINITY, sum = 0.f, x[kCols] = {};
        for (int i = 0; i < pieces; ++i) m = fmaxf(m, ld_cluster(cluster_addr(smem_u32(sst + wrow * 4), i)));
        const float mu = m == -INFINITY ? 0.f : m;
        for (int i = 0; i < pieces; ++i) {
          const float w = ex2(ld_cluster(cluster_addr(smem_u32(sst + wrow * 4), i)) - mu);
          const uint32_t src = cluster_addr(smem_u32(so + wrow * C::kPitch + c0), i);
          sum += w;
#pragma unroll
          for (int c = 0; c < kCols; ++c) x[c] = fmaf(w, ld_cluster(src + 4 * c), x[c]);
        }
        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < kCols; ++c) x[c] *= f;
        store_row<D>(a, sg, own / sg.rts, r, c0, x, sum == 0.f ? -INFINITY : m + log2f(sum));
      }
    }
    cluster_sync();  // no CTA ends while another reads its state
  }
}

// Joins the pieces of an item that parts c, c + 1, ... of the streaming form
// share: LSE = log sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s ("FlashAttention
// -- the same attention, made memory-aware", section 03). Block c has something
// to do when part c begins an item that it does not end. kShare warps per row,
// each taking every kShare-th run of kRun parts with their states all in
// flight: one warp and runs of four for a batch of many items, which have few
// parts each and want small blocks, many to an SM; up to four warps and runs of
// 16 for few items of many parts.
template <int D, int NB, int kShare>
__global__ void __launch_bounds__(256 * NB * kShare) paged_join_kernel(const AttnArgs a) {
  constexpr int R = 8 * NB, kCols = D / 32, kRun = kShare == 1 ? 4 : 16;
  __shared__ float s_x[R][kShare][D];
  __shared__ float s_m[R][kShare], s_sum[R][kShare];
  grid_dep_wait();  // (no early launch of the next kernel: see fa_paged.cuh)
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wrow = warp / kShare, share = warp % kShare;
  const JoinRecord rec = a.records[c];
  if (rec.parts == 0) return;
  const int r = rec.r0 + wrow, last = c + rec.parts - 1;
  const bool live = r < rec.rows;
  float m = -INFINITY, sum = 0.f, x[kCols] = {};
  for (int k0 = c + share * kRun; live && k0 <= last; k0 += kShare * kRun) {
    const int k = k0 + lane;
    const bool on = lane < kRun && k <= last;
    // part c begins the item (piece 1), the others continue it (piece 0)
    const long long at = (static_cast<long long>(k) * 2 + (k == c ? 1 : 0)) * R + wrow;
    const float ls = on ? a.part_lse[at] : -INFINITY;
    float v[kRun][kCols];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      // past the last: part c's state stands in, with weight 0
      const int kj = __shfl_sync(0xffffffffu, on ? k : c, j);
      const float* src = a.part_o + ((static_cast<long long>(kj) * 2 + (kj == c ? 1 : 0)) * R + wrow) * D + lane * kCols;
      if constexpr (kCols == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[j][0] = f.x; v[j][1] = f.y; v[j][2] = f.z; v[j][3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[j][0] = f.x; v[j][1] = f.y;
      }
    }
    float mx = fmaxf(m, ls);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float mu = mx == -INFINITY ? 0.f : mx, alpha = ex2(m - mu);
    const float w = on ? ex2(ls - mu) : 0.f;
    sum *= alpha;
    m = mx;
#pragma unroll
    for (int i = 0; i < kCols; ++i) x[i] *= alpha;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const bool has = __shfl_sync(0xffffffffu, on ? 1 : 0, j) != 0;
      sum += wj;
#pragma unroll
      for (int i = 0; i < kCols; ++i) x[i] = has ? fmaf(wj, v[j][i], x[i]) : x[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i) s_x[wrow][share][lane * kCols + i] = x[i];
  if (lane == 0) {
    s_m[wrow][share] = m;
    s_sum[wrow][share] = sum;
  }
  __syncthreads();
  if (share != 0 || !live) return;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kShare; ++i) m = fmaxf(m, s_m[wrow][i]);
  const float mu = m == -INFINITY ? 0.f : m;
  sum = 0.f;
#pragma unroll
  for (int c2 = 0; c2 < kCols; ++c2) x[c2] = 0.f;
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    const float w = ex2(s_m[wrow][i] - mu);
    sum = fmaf(s_sum[wrow][i], w, sum);
#pragma unroll
    for (int c2 = 0; c2 < kCols; ++c2) x[c2] = fmaf(s_x[wrow][i][lane * kCols + c2], w, x[c2]);
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  const long long at = row_at(a, rec.row0, rec.h, r);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + at * D + lane * kCols);
#pragma unroll
  for (int i = 0; i < kCols; i += 2) dst[i / 2] = pack_bf16(x[i] * f, x[i + 1] * f);
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : kLn2 * (m + log2f(sum));
}

template <int D, int NB, bool kCluster>
int launch_rows(const PagedPool& pool, const AttnArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  using C = Cfg<D, NB>;
  CUtensorMap mk, mv;
  const int box = pool.page_size < C::kTile ? pool.page_size : C::kTile;
  const int blocks = pool.num_pages * pool.num_heads;
  if (!make_map_pages(&mk, pool.k_pages, blocks, pool.page_size, D, box, true) ||
      !make_map_pages(&mv, pool.v_pages, blocks, pool.page_size, D, box, true))
    return -3;
  auto kern = paged_rows_kernel<D, NB, kCluster>;
  // attribute slots 20 to 27
  constexpr int kSlot = 20 + (D == 128 ? 4 : 0) + (NB == 1 ? 2 : 0) + (kCluster ? 1 : 0);
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, kSlot)) return -3;
  const dim3 grid(static_cast<unsigned>(plan.ctas)), block(kThreads);
  cudaError_t e;
  e = launch_clusters(kern, grid, block, C::kSmemBytes, kCluster ? plan.cluster : 1, stream, mk, mv, a);
  if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) return -3;
  if (!kCluster && plan.ctas > 1) {
    // fewer items than SMs: several parts to most of them
    constexpr int kShare = 4 / NB;
    auto join = plan.items < plan.ctas / C::kCtasPerSm ? paged_join_kernel<D, NB, kShare> : paged_join_kernel<D, NB, 1>;
    const int threads = 256 * NB * (plan.items < plan.ctas / C::kCtasPerSm ? kShare : 1);
    e = launch_overlapped(join, dim3(static_cast<unsigned>(plan.ctas - 1)), dim3(threads), 0, stream, a);
    if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) return -3;
  }
  return 0;
}

template <int D>
int launch_rows_d(const PagedPool& pool, const AttnArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  if (plan.cluster > 0)
    return plan.rows == 8 ? launch_rows<D, 1, true>(pool, a, plan, stream) : launch_rows<D, 2, true>(pool, a, plan, stream);
  return plan.rows == 8 ? launch_rows<D, 1, false>(pool, a, plan, stream) : launch_rows<D, 2, false>(pool, a, plan, stream);
}

// What the cluster and the streaming form cost, in microseconds, fitted to the
// times of 350 batch shapes on 152 SMs, of even and of ragged lengths (1 to 64
// sequences of up to 256 to 8192 keys, 2 to 32 key heads, one or a few tokens
// each, no windows): the form chosen is within 2 % of the best one on average. A
// cluster CTA's tiles follow one another, the
// slower the more CTAs share an SM (`more`: CTAs per SM, less one); clusters of
// eight double up on an SM sooner. A streaming CTA has at least kPartUnits
// units, and a second launch joins its pieces. Measured, best cluster / streaming:
// 32 query and 8 key heads, d = 128: 1 x 256 keys 5.4 / 9.3 us, 1 x 4096 9.8 /
// 10.8, 8 x 1024 9.1 / 12.0, but 1 x 8192 14.4 / 12.2 and 32 x 2048 31.5 / 30.2;
// 24 x 5 tokens over 4096 keys, 12 and 4 heads, d = 64: 21.9 / 25.6. One of the
// shapes that the costs misjudge: 16 x 4096, 28.7 / 33.1, streamed.
// The window is left out: the costs count max_kv keys, of which a window shows
// the kernels fewer. 8 x 32768 keys, window 1024: streamed in 11.9 us, clusters
// of two would take 9.2.
struct RowCosts {
  double start, join, more;    // cluster form: one CTA per item, several, and per further CTA of an SM
  double tile, tile_more;      // a tile, and per further CTA of an SM
  double eights;               // SMs that clusters of eight fill before they double up, of all
  double stream, stream_tile;  // streaming form: a launch and its join, and a unit
};
constexpr RowCosts kRowCosts[2][2] = {  // d = 64, 128; 8, 16 rows
    {{2.5, 2, 1.5, 0.80, 0.20, 1.0, 12, 0.90}, {4.0, 2, 3.0, 1.00, 0.40, 1.0, 13, 1.00}},
    {{2.5, 2, 1.6, 0.60, 0.28, 0.6, 10, 0.95}, {3.0, 6, 3.0, 0.72, 0.15, 0.6, 10, 1.00}}};

}  // namespace

PagedPlan paged_attn_plan(const PagedPool& pool, const PagedBatchDev& batch, const int Hq, int max_kv, int sms) {
  PagedPlan r{};
  const long long G = Hq / pool.num_heads;
  const long long rows = batch.max_q * G;
  r.rows = rows <= 8 ? 8 : 16;
  r.row_tiles = static_cast<int>((rows + r.rows - 1) / r.rows);
  const long long items = static_cast<long long>(batch.B) * pool.num_heads * r.row_tiles;
  const int tile = pool.d == 64 ? kTileOf<64> : kTileOf<128>;
  const long long tiles = max_kv > 0 ? (static_cast<long long>(max_kv) + tile - 1) / tile : 1;
  const long long slots = (r.rows == 8 ? 3LL : 2LL) * sms;
  // Chunks (256 rows on the tensor memory; only with more than eight rows): a
  // step of 128 keys costs 1.4 us at d = 64 and 1.6 at d = 128, an item three
  // or four steps more (fa_paged_chunk.cu), a part has eight or more.
  const auto chunk_cost = [&](double pair_items) {
    const double steps = pair_items * (max_kv / 128 + (pool.d == 64 ? 4 : 5)) / sms;
    return pool.d == 64 ? 16 + 1.4 * fmax(steps, 8.0) : 12 + 1.6 * fmax(steps, 8.0);
  };
  const double seqs = batch.B, heads = pool.num_heads;

  // The cluster form, of how many CTAs, or one that needs a workspace? None of
  // what this depends on is the number of packed rows, so that the workspace
  // does not depend on it either.
  const RowCosts& w = kRowCosts[pool.d == 128][r.rows == 16];
  double least = 0;
  for (int c = 1; c <= 8 && items * c <= slots; ++c) {
    const long long per = (tiles + c - 1) / c;
    if (c > 1 && per == (tiles + c - 2) / (c - 1)) continue;  // no fewer tiles per CTA than with one CTA less
    const double more = fmax(static_cast<double>(items * c) / (c > 6 ? w.eights * sms : sms) - 1, 0.0);
    const double cost = w.start + w.more * more + per * (w.tile + w.tile_more * more) + (c > 1 ? w.join : 0);
    if (r.cluster == 0 || cost < least) {
      r.cluster = c;
      least = cost;
    }
  }
  if (r.cluster > 0) {
    const double units = static_cast<double>(items) * (tiles + kItemUnits) / slots;
    if (least < w.stream + w.stream_tile * fmax(units, kPartUnits) &&
        (rows <= 8 || least < chunk_cost(heads * seqs * ((rows + 255) / 256)))) {
      r.ctas = items * r.cluster;
      return r;
    }
    r.cluster = 0;
  }
  // Rows (16 a tile, the cached tiles read once for each) or chunks? Measured,
  // rows streamed / chunks, 32 query and 8 key heads, d = 128: 16 sequences of
  // 2048 keys, 4 tokens each 32 / 44 us; 16 of 512, 16 tokens 32 / 19; 48 of 2048,
  // 8 tokens 103 / 107; 16 and 16 heads, d = 64: 16 of 8192, 32 tokens 135 / 166;
  // 16 of 512, 64 tokens 31 / 27 (misjudged: rows). Over 198 such batches, without
  // windows, the choice is within 1 % of the best form on average. With a window
  // the costs are too high for every form: 4 sequences of 32768 keys, 16 tokens
  // each, 8 heads on one, window 256: chunks in 26 us, a CTA per item would take 9.
  // One form serves the whole call: 63 single tokens over 8192 keys and a chunk
  // of 512 take 472 us together, 161 and 69 in two calls.
  // A ragged batch has at most its packed rows' tiles and one more per sequence.
  const double packed = static_cast<double>(batch.T) * G;
  const double row_items = heads * fmin(seqs * r.row_tiles, seqs + packed / r.rows);
  const double pair_items = heads * fmin(seqs * ((rows + 255) / 256), seqs + packed / 256);
  const double row_cost = w.stream + w.stream_tile * fmax(row_items * (tiles + kItemUnits) / slots, kPartUnits);
  r.chunk = rows > 8 && chunk_cost(pair_items) < row_cost;
  r.ctas = r.chunk ? sms : slots;
  r.items = static_cast<long long>(row_items);
  // The choice depends on the packed rows, what a caller has to provide does not.
  const size_t row_bytes = static_cast<size_t>(slots) * (2 * r.rows * (pool.d + 1) * sizeof(float) + sizeof(JoinRecord));
  const size_t chunk_bytes = rows > 8 ? paged_chunk_workspace_bytes(pool.d, sms) : 0;
  r.workspace_bytes = row_bytes > chunk_bytes ? row_bytes : chunk_bytes;
  return r;
}

int launch_paged_attn(const PagedPool& pool, const PagedBatchDev& batch, const PagedAttn& p,
                      const PagedPlan& plan, void* workspace, cudaStream_t stream) {
  if (plan.chunk) return launch_paged_chunk(pool, batch, p, static_cast<int>(plan.ctas), workspace, stream);
  AttnArgs a{};
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
  a.row_tiles = plan.row_tiles;
  a.cluster = plan.cluster;
  // 0 gives uniform weights: keys that are not seen become -infinity after S has been scaled
  a.scale_log2 = p.scale * kLog2e;
  a.part_o = static_cast<float*>(workspace);
  if (plan.workspace_bytes > 0) {
    a.part_lse = a.part_o + plan.ctas * 2 * plan.rows * pool.d;
    a.records = reinterpret_cast<JoinRecord*>(a.part_lse + plan.ctas * 2 * plan.rows);
  }
  return pool.d == 64 ? launch_rows_d<64>(pool, a, plan, stream) : launch_rows_d<128>(pool, a, plan, stream);
}

}  // namespace fa
