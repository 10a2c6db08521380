// Exact attention over packed sequences with grouped heads: the forward.
//
// Mathematics. Row i of a sequence of n, query head h, key head h / G:
//   s_j = scale q_i . k_j for the keys j that it sees (j <= i if causal, j > i -
//   window if there is one), O = sum_j e^(s_j - m) v_j / l, LSE = m + ln l,
// with the running maximum m and denominator l of fa_fwd.cu, whose key loop this
// is: query tiles resident, key tiles streamed through a TMA ring, S and O in
// tensor memory, P rounded to bf16 for the second product (2^-9 of a weight on
// average), references that move only when passed by 2^8, sums in fp32.
//
// Tiles (fa_packed.cuh): 128 rows are floor(128 / G) tokens with the G heads of
// their key head. At d = 128 a CTA holds two such tiles, which share the stream
// of keys (P over S, 512 tensor-memory columns, one CTA per SM); at d = 64 one,
// with P in columns of its own, and two CTAs share the SM, each filling the
// other's hand-offs: the forms that are fastest without packing as well.
//
// Work. An item is one or two tiles of a sequence with a key head. Where all
// items fit on the GPU at once each CTA finds its own (a call of one short
// prompt is one launch); otherwise persistent CTAs take items from a list,
// heaviest first (make_list). The TMA warp takes them, and leaves a
// record of each for the others, whose barriers run on from item to item.
//
// What a tile's box or the last key tile reaches past its sequence belongs to
// another one. Rows of queries there are not written. Keys there are masked to
// -inf in S, whatever they hold; values there would still be multiplied, by 0,
// which is NaN for what is not finite: the softmax warps, before they hand the
// last tile's P over, put zeros in their place in shared memory.
//
// What bounds it (times of a CUDA graph of the call, replayed back to back; one call
// after another from Python the d = 128 ones take 3 to 5 % more): at d = 128 the tensor
// core, 4 d flops per visible pair (one sequence of 16384 tokens, 32 / 8 heads, causal:
// 1.28 to 1.35 ms as the power limit allows, 1630 to 1715 TFLOP/s, 86 to 90 % of the rate
// of a large library product), less where items are short: 8 prompts of up to 4096
// tokens, 173 us, 73 %. At d = 64 no unit, but the chain of hand-offs from role to role
// (tensor core 39 % busy, issue slots 52 %): 24 images of up to 1369 tokens, 16 heads,
// unmasked, 86.6 us, 41 %; 6 x up to 5001 tokens, 12 / 4 heads, a window of 700, 78 us,
// 33 %, where two or three of seven key tiles are cut by a border.
//
// CTA: softmax warpgroup(s) (thread = row = TMEM lane), an MMA warp, a TMA warp.

#include <algorithm>
#include <limits>

#include "fa_packed.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = kKeyTile;
constexpr int kItems = 4;  // item records kept
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 bf16, 128-byte swizzled
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;  // log2 units that a weight may pass its reference by

// An item, left by the TMA warp.
struct Item {
  int end;          // 1: no more items (the rest is not set)
  int row0, n;      // the sequence's first row, and its length
  int h;            // key head
  int i0;           // token that tile 0 begins with; tile t: i0 + t * tpt
  int j0, ns;       // first key tile, and how many are streamed
  int a[2], m[2];   // tile t takes part in steps [a, a + m)
  int pad;
};

template <int D>
struct Cfg {
  static constexpr int QT = D == 64 ? 1 : 2;  // query tiles
  static constexpr int kCtasPerSm = D == 64 ? 2 : 1;
  static constexpr bool kSepP = D == 64;
  static constexpr int kSoftmaxWarps = 4 * QT;
  static constexpr int kMmaWarp = kSoftmaxWarps, kLoadWarp = kSoftmaxWarps + 1;
  // d = 128: two warps more, which do nothing, complete the warpgroup that gives
  // registers up to the softmax (384 x 168 = 256 x 208 + 128 x 88): spilled values
  // came back from L2, 700 cycles each, at every item's borders.
  static constexpr bool kSplitRegs = D == 128;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + (kSplitRegs ? 4 : 2));
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kStages = 2;
  // d = 64: two buffers of queries, and O is staged in the one that its item is
  // done with; d = 128: one, with room beside it for the staging.
  static constexpr int kQBufs = D == 64 ? 2 : 1;
  static constexpr int kQBytes = QT * kTileBytes;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kQBufs * kQBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kOStageOff = kVOff + kStages * kTileBytes;  // 4 KiB per softmax warp
  static constexpr int kItemOff = kOStageOff + (D == 64 ? 0 : kSoftmaxWarps * 4096);
  static constexpr int kBarOff = kItemOff + kItems * static_cast<int>(sizeof(Item));
  enum : int {
    kBarQFull = 0,
    kBarQFree = kBarQFull + kQBufs,
    kBarKFull = kBarQFree + kQBufs,
    kBarKEmpty = kBarKFull + kStages,
    kBarVFull = kBarKEmpty + kStages,
    kBarVEmpty = kBarVFull + kStages,
    kBarSFull = kBarVEmpty + kStages,  // one per tile from here
    kBarPFull = kBarSFull + QT,
    kBarOFinal = kBarPFull + QT,       // P over S
    kBarSFree = kBarOFinal + QT,       // P apart
    kBarPVDone = kBarSFree + QT,       // P apart
    kBarItemFull = kBarPVDone + QT,
    kBarItemEmpty = kBarItemFull + kItems,
    kBarDrain = kBarItemEmpty + kItems,
    kNumBars
  };
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;  // + slack to align the base
  static constexpr uint32_t kColO = QT * kBN;
  static constexpr uint32_t kColP = kColO + QT * D;  // P apart
  static constexpr uint32_t kTmemCols = D == 64 ? 256 : 512;
  static_assert(kSmemBytes * kCtasPerSm + 1024 * kCtasPerSm <= 233472, "tiles exceed shared memory");
  static_assert(kColP + (kSepP ? QT * 64 : 0) <= kTmemCols, "accumulators exceed tensor memory");
  static_assert(kItemOff % 16 == 0 && sizeof(Item) % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

struct FwdArgs {
  PackedShape s;
  PackedList list;
  __nv_bfloat16* o;  // [T, Hq, d]
  float* lse;        // [T, Hq]
  int* status;
  float scale_log2;
  int boxes;         // 1: a warp's 32 rows are whole tokens, which a box of tmO holds
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtasPerSm)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ FwdArgs args) {
  using C = Cfg<D>;
  constexpr int kS = C::kStages, QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_u32);
  auto bar = [&](int i) -> uint32_t { return base + C::kBarOff + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  volatile int* loaded = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 8);  // stream steps started
  Item* items = reinterpret_cast<Item*>(smem + C::kItemOff);
  const PackedShape& sh = args.s;
  const int G = sh.by_group.G;
  const int warp = warp_id(), lane = lane_id();
  // producer: Q loads and K/V copies started (K of stream step g is copy 2 g, its V 2 g + 1)
  int q_loaded = 0, kv_issued = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(bar(C::kBarQFull + i), 1);
      // every QK^T of the item has completed; d = 64: its O has left the buffer
      mbar_init(bar(C::kBarQFree + i), D == 64 ? C::kSoftmaxWarps : 1);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(bar(C::kBarKFull + i), 1);
      mbar_init(bar(C::kBarKEmpty + i), 1);
      mbar_init(bar(C::kBarVFull + i), 1);
      mbar_init(bar(C::kBarVEmpty + i), 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(bar(C::kBarSFull + t), 1);
      mbar_init(bar(C::kBarPFull + t), 4);  // one arrival per softmax warp
      mbar_init(bar(C::kBarOFinal + t), 1);
      mbar_init(bar(C::kBarSFree + t), 4);
      mbar_init(bar(C::kBarPVDone + t), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(C::kBarItemFull + i), 1);
      mbar_init(bar(C::kBarItemEmpty + i), C::kSoftmaxWarps + 1);
    }
    mbar_init(bar(C::kBarDrain), 1);
    *abort_flag = 0;
    *loaded = 0;
    mbar_fence_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();

  // Hands item number k to a consuming warp; false when the CTA gave up.
  auto get_item = [&](int k, Item* it) -> bool {
    if (!mbar_wait_w(bar(C::kBarItemFull + k % kItems), (k / kItems) & 1, abort_flag)) return false;
    *it = items[k % kItems];
    mbar_arrive_warp(bar(C::kBarItemEmpty + k % kItems));
    return true;
  };

  if (C::kSplitRegs && warp >= C::kSoftmaxWarps) regs_decrease<88>();
  if (warp == C::kLoadWarp) {
    // ------------------------------------------------------------ producer
    ItemQueue queue;
    queue.start(sh, args.list, args.status);
    if (lane == 0) {
      tma_prefetch_map(&tmQ);
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
      const uint32_t q_bytes = static_cast<uint32_t>(sh.tpt * G * 128 * C::kChunks);
      bool ok = true;
      int g = 0, q = 0;
      PackedEntry e;
      int h;
      while (ok && queue.take(&e, &h)) {
        Item it{};
        it.row0 = e.row0;
        it.n = e.n;
        it.h = h;
        it.i0 = e.i0;
        int last = 0;
        int lo[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          const int i = e.i0 + t * sh.tpt;
          const TileRange r = keys_of(sh, e.n, i, min(i + sh.tpt, e.n));
          lo[t] = r.lo;
          it.m[t] = r.n;
          if (r.n > 0) last = r.lo + r.n;  // (a later tile ends no earlier)
        }
        it.j0 = lo[0];  // (nor does it start earlier; tile 0 is never empty)
        it.ns = last - lo[0];
#pragma unroll
        for (int t = 0; t < QT; ++t) it.a[t] = lo[t] - lo[0];
        if (q >= kItems)
          ok = mbar_wait(bar(C::kBarItemEmpty + q % kItems), (q / kItems - 1) & 1, abort_flag);
        if (!ok) break;
        items[q % kItems] = it;
        mbar_arrive(bar(C::kBarItemFull + q % kItems));
        for (int jj = 0; jj < it.ns && ok; ++jj, ++g) {
          const int st = g % kS;
          const uint32_t ph = ((g / kS) + 1) & 1;
          const int key_row = e.row0 + (it.j0 + jj) * kBN;
          queue.step(it.ns - jj);
          if (g >= kS) ok = mbar_wait(bar(C::kBarKEmpty + st), ph, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(C::kBarKFull + st), C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(base + C::kKOff + st * C::kTileBytes + c * kChunkBytes, &tmK, bar(C::kBarKFull + st), c * 64, 0,
                        h, key_row);
          kv_issued = 2 * g + 1;
          if (jj == 0) {
            // this item's queries, once their buffer's item before is done with it
            const int qb = q % C::kQBufs;
            if (q >= C::kQBufs) ok = mbar_wait(bar(C::kBarQFree + qb), (q / C::kQBufs - 1) & 1, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(bar(C::kBarQFull + qb), q_bytes * (QT == 2 && it.m[QT - 1] > 0 ? 2 : 1));
            for (int t = 0; t < QT; ++t) {
              if (it.m[t] == 0) continue;
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_4d(base + C::kQOff + qb * C::kQBytes + t * C::kTileBytes + c * kChunkBytes, &tmQ,
                            bar(C::kBarQFull + qb), c * 64, 0, h, e.row0 + e.i0 + t * sh.tpt);
            }
            q_loaded = ++q;
          }
#ifdef FA_TEST_SKIP_ARRIVE
          // Test-only build (never in libfa.so): the first item's last V tile is
          // never loaded and nothing more is, so the bounded waits for it run out
          // and the CTA winds down through the abort path.
          if (jj == it.ns - 1) {
            ok = false;
            break;
          }
#endif
          if (g >= kS) ok = mbar_wait(bar(C::kBarVEmpty + st), ph, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(C::kBarVFull + st), C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(base + C::kVOff + st * C::kTileBytes + c * kChunkBytes, &tmV, bar(C::kBarVFull + st), c * 64, 0,
                        h, key_row);
          kv_issued = 2 * g + 2;
          *loaded = g + 1;
        }
      }
      if (ok && q >= kItems) ok = mbar_wait(bar(C::kBarItemEmpty + q % kItems), (q / kItems - 1) & 1, abort_flag);
      if (ok) {
        items[q % kItems].end = 1;
        mbar_arrive(bar(C::kBarItemFull + q % kItems));
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // the whole warp runs the issue loop (one elected lane issues)
    constexpr uint32_t kIdS = idesc_bf16_f32(kBM, kBN, false, false);
    constexpr uint32_t kIdO = idesc_bf16_f32(kBM, D, false, true);
    // descriptors built once, advanced by byte offsets / 16
    const uint64_t dQ0 = sdesc_sw128(base + C::kQOff, 16, 1024);
    const uint64_t dK0 = sdesc_sw128(base + C::kKOff, 16, 1024);
    const uint64_t dV0 = sdesc_sw128(base + C::kVOff, kChunkBytes, 1024);
    bool ok = true;
    int k_ready = -1;  // stream steps whose K tile is known to have landed
    auto ensure_k = [&](int gs) {
      if (ok && gs > k_ready) {
        ok = mbar_wait_w(bar(C::kBarKFull + gs % kS), (gs / kS) & 1, abort_flag);
        tc_fence_after();
        k_ready = gs;
      }
    };
    uint64_t dQ = dQ0;
    // S_t = Q_t K^T for stream step gs
    auto issue_s = [&](int t, int gs) {
      const uint64_t qd = dQ + static_cast<uint64_t>((t * C::kTileBytes) >> 4);
      const uint64_t kd = dK0 + static_cast<uint64_t>(((gs % kS) * C::kTileBytes) >> 4);
      mma_ss_depth_w<D>(tmem + t * kBN, qd, kd, kIdS, 0u);
      mma_commit_w(bar(C::kBarSFull + t));
    };
    // O_t (+)= P_t V for stream step gs; P_t (bf16 pairs, 64 columns) over S_t or in its own columns
    auto issue_pv = [&](int t, int gs, bool first) {
      const uint64_t vd = dV0 + static_cast<uint64_t>(((gs % kS) * C::kTileBytes) >> 4);
      const uint32_t pcol = C::kSepP ? C::kColP + t * 64 : t * kBN;
      mma_ts_depth_w<false>(tmem + C::kColO + t * D, tmem + pcol, vd, kIdO, first ? 0u : 1u);
    };
    int g = 0;
    int ut[QT] = {};  // S tiles of tile t over all items (its S/P barrier phases)
    Item it;
    for (int q = 0; ok; ++q) {
      ok = get_item(q, &it);
      if (!ok || it.end) break;
      const int ns = it.ns, qb = q % C::kQBufs;
      dQ = dQ0 + static_cast<uint64_t>((qb * C::kQBytes) >> 4);
      ok = mbar_wait_w(bar(C::kBarQFull + qb), (q / C::kQBufs) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if constexpr (C::kSepP) {
        // S for the step, once its predecessor is in the softmax's registers
        auto next_s = [&](int gs, int s_issued) {
          if (s_issued > 0) ok = mbar_wait_w(bar(C::kBarSFree), (s_issued - 1) & 1, abort_flag);
          ensure_k(gs);
          if (!ok) return;
          tc_fence_after();
          issue_s(0, gs);
          mma_commit_w(bar(C::kBarKEmpty + gs % kS));
        };
        next_s(g, ut[0]);
        for (int jj = 0; jj < ns && ok; ++jj) {
          const int gs = g + jj;
          // the next step's QK^T first, so that it computes while the softmax forms P
          if (jj + 1 < ns) next_s(gs + 1, ut[0] + 1);
          if (!ok) break;
          ok = mbar_wait_w(bar(C::kBarVFull + gs % kS), (gs / kS) & 1, abort_flag);
          if (ok) ok = mbar_wait_w(bar(C::kBarPFull), ut[0] & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, gs, jj == 0);
          mma_commit_w(bar(C::kBarPVDone));
          mma_commit_w(bar(C::kBarVEmpty + gs % kS));
          ++ut[0];
        }
      } else {
        // the item's first QK^T goes behind the previous item's last P.V (in
        // order on the tensor core, so that P.V has read P before S lands there)
        ensure_k(g);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < QT; ++t)
          if (it.m[t] > 0 && it.a[t] == 0) issue_s(t, g);
        mma_commit_w(bar(C::kBarKEmpty + g % kS));
        if (ns == 1) mma_commit_w(bar(C::kBarQFree));
        for (int jj = 0; jj < ns && ok; ++jj) {
          const int gs = g + jj;
          ok = mbar_wait_w(bar(C::kBarVFull + gs % kS), (gs / kS) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            const int u = jj - it.a[t];  // tile-local step
            if (!ok || u < 0 || u >= it.m[t]) continue;
            ok = mbar_wait_w(bar(C::kBarPFull + t), ut[t] & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, gs, u == 0);
            ++ut[t];
            if (u + 1 < it.m[t]) {
              ensure_k(gs + 1);
              if (!ok) break;
              issue_s(t, gs + 1);
            } else {
              mma_commit_w(bar(C::kBarOFinal + t));
            }
          }
          if (!ok) break;
          // a tile whose range starts at the next step (a window's later start)
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            if (!ok || it.m[t] == 0 || it.a[t] != jj + 1) continue;
            ensure_k(gs + 1);
            if (!ok) break;
            issue_s(t, gs + 1);
          }
          if (!ok) break;
          // every QK^T of the item has been issued: its Q buffer is free once they complete
          if (jj == ns - 2) mma_commit_w(bar(C::kBarQFree));
          mma_commit_w(bar(C::kBarVEmpty + gs % kS));
          if (jj + 1 < ns) mma_commit_w(bar(C::kBarKEmpty + (gs + 1) % kS));
        }
      }
      g += ns;
    }
    // Let every MMA this warp issued finish before TMEM is released.
    mma_commit_w(bar(C::kBarDrain));
    mbar_wait_w(bar(C::kBarDrain), 0, nullptr);
  } else if (warp < C::kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    if constexpr (C::kSplitRegs) regs_increase<208>();
    const int t = warp / 4;  // query tile
    const int r = threadIdx.x & 127;  // row of the tile
    const int ri = sh.by_group.div(r);  // its token
    // tokens of the warp's first and last rows
    const int warp_i0 = sh.by_group.div(r - lane), warp_i1 = sh.by_group.div(r - lane + 31);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * kBN;
    const uint32_t tO = tmem + lane_base + C::kColO + t * D;
    const uint32_t tP = tmem + lane_base + C::kColP + t * 64;  // P apart
    const float sl2 = args.scale_log2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    bool ok = true;
    int g = 0;           // stream steps before this item
    int ut = 0, qt = 0;  // S tiles and items of this query tile so far
    for (int q = 0; ok; ++q) {
      // (the record is given back at the item's end: what the loop does not need is read again there)
      if constexpr (QT == 1)
        ok = mbar_wait_w(bar(C::kBarItemFull + q % kItems), (q / kItems) & 1, abort_flag);
      else  // (a whole item, where this tile of the last one held no rows)
        ok = mbar_wait_long_w(bar(C::kBarItemFull + q % kItems), (q / kItems) & 1, abort_flag, loaded);
      if (!ok) break;
      const Item& it = items[q % kItems];
      if (it.end) break;
      const int n_mine = it.m[t], n = it.n;
      int gs = g + it.a[t], key0 = (it.j0 + it.a[t]) * kBN;
      g += it.ns;
      if (n_mine == 0) {
        mbar_arrive_warp(bar(C::kBarItemEmpty + q % kItems));
        continue;
      }
      // keys visible to this row: key_lo <= key < key_hi; to all rows of the warp: full_lo <= key < full_hi
      int key_hi = n, key_lo = 0, full_hi = n, full_lo = 0;
      {
        const int i0 = it.i0 + t * sh.tpt, pos = i0 + ri;
        if (sh.causal) {
          key_hi = min(n, pos + 1);
          full_hi = min(n, i0 + warp_i0 + 1);
        }
        if (sh.window > 0) {
          key_lo = pos - sh.window + 1;
          full_lo = i0 + warp_i1 - sh.window + 1;
        }
      }
      float m_ref = -INFINITY;  // log2-domain reference maximum
      float l = 0.f;
      for (int u = 0; u < n_mine; ++u, ++ut, ++gs, key0 += kBN) {
        ok = mbar_wait_w(bar(C::kBarSFull + t), ut & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
        if constexpr (C::kSepP) {  // S is in registers: the next QK^T may overwrite it
          tc_fence_before();
          mbar_arrive_warp(bar(C::kBarSFree + t));
        }
        float xs[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) xs[c] = __uint_as_float(sr[c >> 5][c & 31]);
        // masks, by words of 32 keys, where a border of some row of the warp cuts the
        // tile. (Little code, here and below, rather than few instructions: the hot
        // loops of all roles share the instruction cache. A comparison per key and
        // border took 4 % more, 6 x up to 5001 tokens, window 700, d = 64.)
        if (key0 + kBN > full_hi || key0 < full_lo) {
          const int hi = key_hi - key0, lo = key_lo - key0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int h = hi - 32 * w, l = lo - 32 * w;
            uint32_t keep = h >= 32 ? 0xffffffffu : (1u << max(h, 0)) - 1u;
            keep &= l >= 32 ? 0u : 0xffffffffu << max(l, 0);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(keep & (1u << c))) xs[32 * w + c] = -INFINITY;
          }
        }
        const float m_tile = max3(fmaxf(max32(xs), max32(xs + 32)), max32(xs + 64), max32(xs + 96)) * sl2;
        const bool need = m_tile > m_ref + kSlack;
        const float m_old = m_ref;
        if (need) m_ref = m_tile;
        const float alpha = need ? ex2(m_old - m_ref) : 1.0f;
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        // p = exp2(s * scale * log2(e) - m_ref), packed two at a time; P
        // columns [32 h, 32 h + 32) hold scores [64 h, 64 h + 64), over S or
        // in P's own columns once the previous P.V has read them
        const float2 negm = make_float2(-m_use, -m_use);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[32];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int x = 64 * hf + 2 * c;
            const float2 a = __ffma2_rn(make_float2(xs[x], xs[x + 1]), sl2x2, negm);
            const float2 pr = make_float2(ex2(a.x), ex2(a.y));
            if (c & 1) acc1 = __fadd2_rn(acc1, pr);
            else acc0 = __fadd2_rn(acc0, pr);
            pk[c] = pack_bf16(pr.x, pr.y);
          }
          if constexpr (C::kSepP) {
            if (hf == 0 && ut > 0) {
              ok = mbar_wait_w(bar(C::kBarPVDone + t), (ut - 1) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
            }
            tmem_st32(tP + 32 * hf, pk);
          } else {
            tmem_st32(tS + 32 * hf, pk);
          }
        }
        if (!ok) break;
        l = alpha * l + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
        // Rescale the accumulator when this warp's maximum moved. O is
        // settled: this S was committed after the tile's previous P.V (P over
        // S), or that P.V's completion was waited for above (P apart).
        if (u > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1  // (unrolled: 176 instead of 173 us, 8 prompts of up to 4096 tokens, d = 128)
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
            const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), al2);
              o[x] = __float_as_uint(v.x);
              o[x + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + c * 32, o);
          }
        }
        if (key0 + kBN > n) {
          // values past the sequence: zeros (both tiles may write them, and one
          // while the other's P.V reads them: they are zeros by then already)
          const int st = gs % kS;
          ok = mbar_wait_w(bar(C::kBarVFull + st), (gs / kS) & 1, abort_flag);
          if (!ok) break;
          zero_rows(smem + C::kVOff + st * C::kTileBytes, kChunkBytes, C::kChunks, n - key0, kBN, r, 128);
          fence_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(bar(C::kBarPFull + t));
      }
      if (!ok) break;
      // write-back once the item's last P.V for this tile has completed; the
      // tile's next P.V (next item) waits for this warpgroup's next P, so O is
      // read out before it is overwritten
      if constexpr (C::kSepP)
        ok = mbar_wait_w(bar(C::kBarPVDone + t), (ut - 1) & 1, abort_flag);
      else
        ok = mbar_wait_w(bar(C::kBarOFinal + t), qt & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const float inv_l = l == 0.f ? 0.f : 1.0f / l;  // (NaN stays NaN)
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      const float lse_row = l == 0.f ? -INFINITY : (m_use + log2f(l)) * kLn2;
      const float2 il2 = make_float2(inv_l, inv_l);
      // Each warp swizzles its 32 rows, 64 columns at a time, into its staging
      // block. At d = 128, where they are all the sequence's and whole tokens, one
      // tensor copy takes them from there while the warp goes on (an SM's own stores
      // move 32 bytes a clock: 2000 cycles an item; 8 prompts of up to 4096 tokens,
      // 32 / 8 heads: 173 us, not 180. At d = 64 the other CTA has the tensor core
      // meanwhile, and nothing was gained.) Otherwise the warp writes them back as
      // four whole lines per instruction.
      const int i0 = it.i0 + t * sh.tpt;
      const long long first = static_cast<long long>(it.row0 + i0) * sh.Hq + it.h * G;  // (token, head) of row 0
      const bool box = D == 128 && args.boxes && i0 + warp_i1 < n;
      uint8_t* stage_blk = smem + (D == 64 ? C::kQOff + (q % C::kQBufs) * C::kQBytes : C::kOStageOff) + warp * 4096;
      uint8_t* stage_row = stage_blk + lane * 128;
#pragma unroll 1
      for (int h = 0; h < D / 64; ++h) {
        uint32_t pko[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + h * 64 + c * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), il2);
            pko[16 * c + e] = pack_bf16(v.x, v.y);
          }
        }
        if constexpr (D == 128) {  // the block's last copy has read it
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        }
        // 16-byte chunk v of row `lane` in slot v ^ (lane & 7)
#pragma unroll
        for (int v = 0; v < 8; ++v)
          *reinterpret_cast<uint4*>(stage_row + ((v ^ (lane & 7)) * 16)) =
              make_uint4(pko[4 * v], pko[4 * v + 1], pko[4 * v + 2], pko[4 * v + 3]);
        if (box) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&tmO, smem_u32(stage_blk), h * 64, 0, it.h, it.row0 + i0 + warp_i0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          // instruction j: lanes 8r'..8r'+7 write the eight chunks of row 4j + r'
          uint4 val[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int wr = 4 * j + (lane >> 3), v = lane & 7;
            val[j] = *reinterpret_cast<const uint4*>(stage_blk + wr * 128 + ((v ^ (wr & 7)) * 16));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = (warp & 3) * 32 + 4 * j + (lane >> 3), x = sh.by_group.div(row);
            if (x < sh.tpt && i0 + x < n)
              *reinterpret_cast<uint4*>(args.o + (first + static_cast<long long>(x) * sh.Hq + (row - x * G)) * D + h * 64 +
                                        (lane & 7) * 8) = val[j];
          }
          __syncwarp();  // the block is read back before it is written again
        }
      }
      if (ri < sh.tpt && i0 + ri < n) args.lse[first + static_cast<long long>(ri) * sh.Hq + (r - ri * G)] = lse_row;
      mbar_arrive_warp(bar(C::kBarItemEmpty + q % kItems));
      if constexpr (D == 64) {  // the next item but one may load its queries here
        fence_async_smem();
        mbar_arrive_warp(bar(C::kBarQFree + q % C::kQBufs));
      }
      ++qt;
    }
    if (D == 128 && lane == 0) bulk_wait<0>();  // this warp's copies out of shared memory
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kLoadWarp && lane == 0 && *abort_flag) {
    // Every role has stopped, so the flag is final: let every copy this thread
    // started land before the CTA exits (only the last load of each buffer and
    // the last 2 x stages K/V copies can still be pending).
    for (int i = max(q_loaded - C::kQBufs, 0); i < q_loaded; ++i)
      mbar_wait(bar(C::kBarQFull + i % C::kQBufs), (i / C::kQBufs) & 1, nullptr);
    for (int c = kv_issued - 1; c >= 0 && c >= kv_issued - 2 * kS; --c) {
      const int gg = c >> 1, st = gg % kS;
      mbar_wait(bar(((c & 1) ? C::kBarVFull : C::kBarKFull) + st), (gg / kS) & 1, nullptr);
    }
  }
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(args.status, kStatusTimeout);
}

// Entries of a call at most, and whether it needs a list: not where each item has a CTA.
struct FwdPlan {
  int unit, cap;
  int slots;  // CTAs that run at once
  bool listed;
};

FwdPlan fwd_plan(int B, int T, int Hq, int Hkv, int d, int sms) {
  FwdPlan p;
  const int qt = d == 64 ? 1 : 2;
  p.unit = 128 / (Hq / Hkv) * qt;
  p.cap = T / p.unit + B;
  p.slots = sms * (d == 64 ? 2 : 1);
  p.listed = static_cast<long long>(p.cap) * Hkv > p.slots;
  return p;
}

template <int D>
int launch_d(const PackedProblem& p, const FwdArgs& a, const FwdPlan& plan, cudaStream_t stream) {
  using C = Cfg<D>;
  const PackedShape& s = p.s;
  const int G = s.by_group.G;
  CUtensorMap mq, mk, mv, mo;
  FwdArgs args = a;
  args.boxes = D == 128 && 32 % G == 0;
  if (!make_map_packed(&mq, p.q, s.T, s.Hkv, G, D, p.q_stride, s.tpt) ||
      !make_map_packed(&mk, p.k, s.T, s.Hkv, 1, D, p.k_stride, kBN) ||
      !make_map_packed(&mv, p.v, s.T, s.Hkv, 1, D, p.v_stride, kBN) ||
      !make_map_packed(&mo, a.o, s.T, s.Hkv, G, D, static_cast<long long>(s.Hq) * D, args.boxes ? 32 / G : 1))
    return -3;
  auto kern = packed_fwd_kernel<D>;
  // attribute slots 30 and 31 (the other kernels use 0-29)
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, D == 64 ? 30 : 31)) return -3;
  const int grid = plan.listed ? plan.slots : plan.cap * s.Hkv;
  const cudaError_t e = launch_overlapped(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, stream, mq, mk, mv, mo, args);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace

size_t packed_fwd_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int sms) {
  const FwdPlan p = fwd_plan(B, T, Hq, Hkv, d, sms);
  return p.listed ? sizeof(PackedHead) + static_cast<size_t>(p.cap) * sizeof(int4) : 0;
}

int launch_packed_fwd(const PackedProblem& p, void* o, float* lse, void* workspace, cudaStream_t stream) {
  const PackedShape& s = p.s;
  const int sms = device_sm_count();
  FwdArgs a{};
  a.s = s;
  a.status = device_status_word();
  if (!a.status || sms <= 0) return -3;
  const FwdPlan plan = fwd_plan(s.B, s.T, s.Hq, s.Hkv, p.d, sms);
  a.list = PackedList{static_cast<PackedHead*>(workspace), nullptr, plan.cap, plan.unit, 1, 0};
  if (plan.listed) {
    a.list.entries = reinterpret_cast<int4*>(a.list.head + 1);
    const int rc = launch_packed_plan(s, a.list, stream);
    if (rc != 0) return rc;
  }
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  // 0 would make NaN of the -infinity of a masked key. The least there is, 2^-149,
  // leaves scores below 2^-21: all weights alike, as they are to be.
  a.scale_log2 = std::max(p.scale * kLog2e, std::numeric_limits<float>::denorm_min());
  return p.d == 64 ? launch_d<64>(p, a, plan, stream) : launch_d<128>(p, a, plan, stream);
}

}  // namespace fa
