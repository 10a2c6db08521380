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
// (2^-12) and scaled by 2^15, so that weights down to 2^-29 of the largest
// keep full precision and down to 2^-39 are not lost. The denominator adds
// the weights before that rounding.
//
// What bounds it: at one token per sequence every cached byte is read once
// for G = Hq / Hkv rows of arithmetic, far below the tensor core's rate, so
// the kernel is a copy from HBM. It therefore is organised as one: a TMA warp
// keeps a ring of tiles (64 tokens of K and V) full, as deep as two CTAs per
// SM allow, and four warps take 16 tokens of each tile, each with an online
// softmax of its own, so that no two warps wait for one another until the
// end. Codes go from shared memory to registers and are widened there
// (mma.sync takes its operands from registers; tcgen05 would want them
// widened in shared memory first, which costs a second pass over it).

#include <cmath>

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kTile = 64;        // tokens per stage
constexpr int kGroup = 16;       // tokens per warp of a stage
constexpr int kRows = 16;        // query rows per CTA
constexpr int kThreads = 160;    // four warps and the TMA warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 15.f;  // P is held as 2^15 P

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 6 : 10;  // two CTAs per SM
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kStages * kTileBytes;
  static constexpr int kScaleOff = 2 * kStages * kTileBytes;  // [stage][4] {sk, log2 sv}
  static constexpr int kBarOff = kScaleOff + kStages * 4 * 8;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;  // + slack to align the base
  // the warps' states at the end, in the ring's place
  static constexpr int kPitch = D + 4;
  static_assert(4 * kRows * (kPitch + 4) * 4 <= kScaleOff, "the warps' states must fit the ring");
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

struct AttnArgs {
  PagedBatchDev batch;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [item][split][16][d], normalised
  float* part_lse;  // [item][split][16], log2 units
  const uint8_t* v_pages;  // the rare path that looks for NaN codes again
  const float* k_scales;
  const float* v_scales;
  int* status;
  int Hq, Hkv, G;
  int window;
  int row_tiles, splits, split_tiles;
  float scale_log2;
};

// The rows of one CTA (16 of the n * G rows of a sequence and key head, query
// by query) and the keys that they see.
struct RowTile {
  int rows, r0;
  int p0;          // position of query 0
  int p_lo, p_hi;  // positions of the first and last query of the tile
  int lo, hi;      // keys that any of its rows sees: [lo, hi)
  int t0, nt;      // as tiles of 64
  int active;      // splits with work
};

__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, const PagedSeq& s, int rt) {
  RowTile g;
  g.rows = s.n * a.G;
  g.r0 = rt * kRows;
  g.p0 = s.len - s.n;
  g.p_lo = g.p0 + g.r0 / a.G;
  g.p_hi = g.p0 + (min(g.r0 + kRows, g.rows) - 1) / a.G;
  g.hi = max(g.p_hi + 1, 0);
  g.lo = a.window > 0 ? max(g.p_lo - a.window + 1, 0) : 0;
  g.t0 = g.lo / kTile;
  g.nt = g.hi > g.lo ? (g.hi + kTile - 1) / kTile - g.t0 : 0;
  g.active = min((g.nt + a.split_tiles - 1) / a.split_tiles, a.splits);
  return g;
}

__device__ __forceinline__ bool sees(int p, int j, int window) {
  return j <= p && (window == 0 || j > p - window);
}

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

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// One row's D/4 consecutive queries of this lane, scaled into f16, and the
// factor that undoes it (with the softmax scale). Four words of eight values
// per 16 bytes; word pairs are the two halves of an mma step's A columns.
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

// kHalf: at most eight rows, the upper half of every m16 tile is zero and its
// softmax left out.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const AttnArgs a) {
  using C = Cfg<D>;
  constexpr int kS = C::kStages;
  constexpr int kNR = kHalf ? 1 : 2;  // row halves per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const uint32_t full = sb + C::kBarOff, empty = full + 8 * kS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* nan_flag = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 4);
    }
    *abort_flag = 0;
    *nan_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();

  const int split = static_cast<int>(blockIdx.x % a.splits);
  const long long item = blockIdx.x / a.splits;
  const int rt = static_cast<int>(item % a.row_tiles);
  const long long bh = item / a.row_tiles;
  const int h = static_cast<int>(bh % a.Hkv), seq = static_cast<int>(bh / a.Hkv);
  const PagedSeq s = paged_seq(a.batch, seq, a.status);
  if (rt * kRows >= s.n * a.G) return;
  const RowTile g = row_tile(a, s, rt);
  if (split >= max(g.active, 1)) return;
  const int ta = g.t0 + split * a.split_tiles;
  const int tb = split == g.active - 1 ? g.t0 + g.nt : min(ta + a.split_tiles, g.t0 + g.nt);
  const int tiles = g.nt > 0 ? tb - ta : 0;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA warp
    // Lane i looks up the i-th of the next 32 groups of 16 keys: its page and
    // scales, two dependent loads that are paid once for eight tiles.
    const int box_rows = min(a.batch.page_size, kTile);
    const int boxes = kTile / box_rows, groups_per_box = box_rows / kGroup;
    int armed = 0;
    for (int base = 0; base < tiles && !*abort_flag; base += 8) {
      int page = -1;
      float sk = -1.f, ev = 0.f;
      const int j0 = (ta + base) * kTile + lane * kGroup;
      if (base + lane / 4 < tiles && j0 < g.hi && j0 + kGroup > g.lo) {
        page = paged_page(a.batch, seq, j0 >> a.batch.page_shift, a.status);
        if (page >= 0) {
          const long long at = static_cast<long long>(page) * a.Hkv + h;
          sk = a.k_scales[at];
          const float sv = a.v_scales[at];
          const uint32_t bits = __float_as_uint(sv);
          // exact for the powers of two that the append writes
          ev = (bits & 0x7fffffu) ? log2f(sv) : bits == 0 ? -INFINITY : static_cast<float>(static_cast<int>(bits >> 23) - 127);
        }
      }
      for (int i = 0; i < 8 && base + i < tiles; ++i) {
        const int it = base + i, st = it % kS;
        int pg[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) pg[q] = __shfl_sync(0xffffffffu, page, 4 * i + q);
        if (it >= kS && !mbar_wait_w(empty + 8 * st, (it / kS - 1) & 1, abort_flag)) break;
        if (lane / 4 == i)
          *reinterpret_cast<float2*>(smem + C::kScaleOff + (st * 4 + (lane & 3)) * 8) = make_float2(sk, ev);
        __syncwarp();
        if (lane == 0) {
          int n = 0;
          int bp[4];
          for (int b = 0; b < boxes; ++b) {
            bp[b] = -1;
            for (int q = 0; q < groups_per_box; ++q) bp[b] = max(bp[b], pg[b * groups_per_box + q]);
            n += bp[b] >= 0;
          }
          mbar_arrive_expect_tx(full + 8 * st, 2u * n * box_rows * D);
          const int tok = (ta + it) * kTile;
          for (int b = 0; b < boxes; ++b) {
            if (bp[b] < 0) continue;
            const int slot = (tok + b * box_rows) & (a.batch.page_size - 1);
            const int blk = bp[b] * a.Hkv + h;
            const uint32_t off = st * C::kTileBytes + b * box_rows * D;
            tma_load_3d(sb + C::kKOff + off, &tmK, full + 8 * st, 0, slot, blk);
            tma_load_3d(sb + C::kVOff + off, &tmV, full + 8 * st, 0, slot, blk);
          }
        }
        armed = it + 1;
      }
      __syncwarp();
    }
    // let every copy in flight land before the CTA can end
    for (int it = max(armed - kS, 0); it < armed; ++it) mbar_wait(full + 8 * (it % kS), (it / kS) & 1, nullptr);
    if (lane == 0 && *abort_flag) *a.status = kStatusTimeout;
    return;
  }

  // -------------------------------------------------------------- four compute warps
  const int n = lane >> 2, t = lane & 3;  // fragment row (or column) and quarter
  uint32_t qa[D / 16][4];
  float qf[2];
  int p_row[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = g.r0 + n + 8 * r;
    const bool on = row < g.rows && (r == 0 || !kHalf);
    const int i = on ? row / a.G : 0, hd = h * a.G + (on ? row % a.G : 0);
    p_row[r] = on ? g.p0 + i : g.p_hi;
    uint32_t w[D / 8];
    qf[r] = load_query<D>(a.q + static_cast<long long>(s.row0 + i) * a.q_stride + hd * D + t * (D / 4), on,
                          a.scale_log2, w);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qa[k][r] = w[2 * k];
      qa[k][2 + r] = w[2 * k + 1];
    }
  }
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ms[2] = {-INFINITY, -INFINITY}, mt[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  bool ok = true, saw_nan = false;

  for (int it = 0; it < tiles; ++it) {
    const int st = it % kS;
    ok = mbar_wait_w(full + 8 * st, (it / kS) & 1, abort_flag);
    if (!ok) break;
    const float2 sc = *reinterpret_cast<const float2*>(smem + C::kScaleOff + (st * 4 + warp) * 8);
    if (!(sc.x < 0.f)) {  // below zero: no row sees these keys, or they have no page
      const int j0 = (ta + it) * kTile + warp * kGroup;
      const bool part = !all_see(g, j0, a.window);
      const uint8_t* kb = smem + C::kKOff + st * C::kTileBytes;
      const uint8_t* vb = smem + C::kVOff + st * C::kTileBytes;
      // S = Q K^T: 16 rows x 16 keys. A lane holds D/4 consecutive channels of
      // its key, four per mma step, in the order that its queries have.
      float acc[2][4] = {};
      uint4 kw[2][D / 64];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int row = warp * kGroup + nb * 8 + n;
        if constexpr (D == 128) {
          kw[nb][0] = *reinterpret_cast<const uint4*>(kb + row * 128 + (((2 * t) ^ (row & 7)) << 4));
          kw[nb][1] = *reinterpret_cast<const uint4*>(kb + row * 128 + (((2 * t + 1) ^ (row & 7)) << 4));
        } else {
          kw[nb][0] = *reinterpret_cast<const uint4*>(kb + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
        }
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const uint32_t w = e == 0 ? kw[nb][c].x : e == 1 ? kw[nb][c].y : e == 2 ? kw[nb][c].z : kw[nb][c].w;
            mma16816(acc[nb], qa[4 * c + e], e4m3x2_to_f16x2(static_cast<uint16_t>(w)),
                     e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)));
          }
        }
      }
      uint32_t pa[4] = {0u, 0u, 0u, 0u};
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int r = 0; r < kNR; ++r) {
        const float f = qf[r] * sc.x;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = acc[e >> 1][2 * r + (e & 1)] * f;
          if (part && !sees(p_row[r], j0 + (e >> 1) * 8 + 2 * t + (e & 1), a.window)) x[e] = -INFINITY;
        }
        const float mx = quad_max(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
        const float ms_new = fmaxf(ms[r], mx), mt_new = fmaxf(mt[r], mx + sc.y);
        // a row that has seen nothing yet has both at -infinity
        const float su = ms_new == -INFINITY ? 0.f : ms_new, tu = mt_new == -INFINITY ? 0.f : mt_new;
        const float ls = ex2(ms[r] - su);
        alpha[r] = ex2(mt[r] - tu);
        const float f2 = ex2(fminf(su + sc.y - tu + kPShift, 126.f));
        float p[4], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(x[e] - su);
          sum += p[e];
        }
        l[r] = fmaf(l[r], ls, sum);
        ms[r] = ms_new;
        mt[r] = mt_new;
        pa[r] = pack_f16(p[0] * f2, p[1] * f2);
        pa[2 + r] = pack_f16(p[2] * f2, p[3] * f2);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || (!kHalf && alpha[1] != 1.f))) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          if constexpr (!kHalf) {
            o[i][2] *= alpha[1];
            o[i][3] *= alpha[1];
          }
        }
      }
      // O += P V: lane (n, t) takes channels [n D/8, (n + 1) D/8) of keys 2t, 2t+1, 2t+8, 2t+9
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = warp * kGroup + 2 * t + (e & 1) + 8 * (e >> 1);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(vb + row * 128 + ((n ^ (row & 7)) << 4));
          vw[e][0] = w.x; vw[e][1] = w.y; vw[e][2] = w.z; vw[e][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vb + row * 64 + (((n >> 1) ^ ((row >> 1) & 3)) << 4) +
                                                          ((n & 1) << 3));
          vw[e][0] = w.x; vw[e][1] = w.y;
        }
      }
      if (part) {
        // keys that a row does not see have weight 0, and 0 x NaN is NaN: here
        // NaN codes are taken out, and rows that do see one are mended at the end
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t z = nan_bytes(vw[e][i]);
            saw_nan = saw_nan || z != 0;
            vw[e][i] &= ~z;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // byte pairs of two neighbouring keys, channel by channel
        const uint32_t a01 = __byte_perm(vw[0][i], vw[1][i], 0x5140), a23 = __byte_perm(vw[0][i], vw[1][i], 0x7362);
        const uint32_t b01 = __byte_perm(vw[2][i], vw[3][i], 0x5140), b23 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
        mma16816(o[4 * i], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a01)), e4m3x2_to_f16x2(static_cast<uint16_t>(b01)));
        mma16816(o[4 * i + 1], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a01 >> 16)),
                 e4m3x2_to_f16x2(static_cast<uint16_t>(b01 >> 16)));
        mma16816(o[4 * i + 2], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a23)), e4m3x2_to_f16x2(static_cast<uint16_t>(b23)));
        mma16816(o[4 * i + 3], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(a23 >> 16)),
                 e4m3x2_to_f16x2(static_cast<uint16_t>(b23 >> 16)));
      }
    }
    mbar_arrive_warp(empty + 8 * st);
  }
  if (saw_nan) *nan_flag = 1;

  // -------------------------------------------------------------- join the four warps
  named_bar_sync(1, 128);  // every warp is done with the ring
  if (*abort_flag) {
    if (threadIdx.x == 0) *a.status = kStatusTimeout;
    return;  // all 128 threads alike: the flag is only raised by a wait, and all waits are over
  }
  float* so = reinterpret_cast<float*>(smem);               // [warp][row][kPitch]
  float* sst = so + 4 * kRows * C::kPitch;                  // [warp][row][4]: m_s, m_t, l
#pragma unroll
  for (int r = 0; r < kNR; ++r) {
    const int row = n + 8 * r;
    const float sum = quad_sum(l[r]);
    float* dst = so + (warp * kRows + row) * C::kPitch + t * (D / 4);
    // o[i][2r + e] is channel (D/8) (2t + e) + i
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < D / 8; i += 4)
        *reinterpret_cast<float4*>(dst + e * (D / 8) + i) =
            make_float4(o[i][2 * r + e], o[i + 1][2 * r + e], o[i + 2][2 * r + e], o[i + 3][2 * r + e]);
    if (t == 0) {
      float* st = sst + (warp * kRows + row) * 4;
      st[0] = ms[r];
      st[1] = mt[r];
      st[2] = sum;
    }
  }
  named_bar_sync(1, 128);
  constexpr int kCols = D / 8;  // per thread, eight threads per row
  const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * kCols;
  if (g.r0 + row >= g.rows) return;
  float m = -INFINITY, mv = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    m = fmaxf(m, sst[(w * kRows + row) * 4]);
    mv = fmaxf(mv, sst[(w * kRows + row) * 4 + 1]);
  }
  const float mu = m == -INFINITY ? 0.f : m, vu = mv == -INFINITY ? 0.f : mv;
  float sum = 0.f, x[kCols] = {};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float* st = sst + (w * kRows + row) * 4;
    sum += st[2] * ex2(st[0] - mu);
    const float f = ex2(st[1] - vu);
    const float* src = so + (w * kRows + row) * C::kPitch + c0;
#pragma unroll
    for (int i = 0; i < kCols; ++i) x[i] = fmaf(src[i], f, x[i]);
  }
  // sum = 0: the row saw no key
  const float f = sum == 0.f ? 0.f : ex2(vu - mu - kPShift) / sum;
#pragma unroll
  for (int i = 0; i < kCols; ++i) x[i] *= f;
  const int qi = (g.r0 + row) / a.G, hd = h * a.G + (g.r0 + row) % a.G;
  if (*nan_flag) {
    const int p = g.p0 + qi;
    for (int j = max(ta * kTile, g.lo); j < min(tb * kTile, g.hi); ++j) {
      if (all_see(g, j & ~(kGroup - 1), a.window) || !sees(p, j, a.window)) continue;
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
  if (g.active > 1) {
    const long long at = (item * a.splits + split) * kRows + row;
    float* dst = a.part_o + at * D + c0;
#pragma unroll
    for (int i = 0; i < kCols; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    if (c0 == 0) a.part_lse[at] = sum == 0.f ? -INFINITY : m + log2f(sum);
    return;
  }
  const long long at = static_cast<long long>(s.row0 + qi) * a.Hq + hd;
  uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + c0);
#pragma unroll
  for (int i = 0; i < kCols; i += 8)
    dst[i / 8] = make_uint4(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]),
                            pack_bf16(x[i + 4], x[i + 5]), pack_bf16(x[i + 6], x[i + 7]));
  if (c0 == 0) a.lse[at] = sum == 0.f ? -INFINITY : kLn2 * (m + log2f(sum));
}

// Joins the splits' states of 16 rows: LSE = log sum_s exp(LSE_s), O = sum_s
// exp(LSE_s - LSE) O_s ("FlashAttention -- the same attention, made
// memory-aware", section 03). Eight threads per row.
template <int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const AttnArgs a) {
  constexpr int kCols = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const long long item = blockIdx.x;
  const int rt = static_cast<int>(item % a.row_tiles);
  const long long bh = item / a.row_tiles;
  const int h = static_cast<int>(bh % a.Hkv), seq = static_cast<int>(bh / a.Hkv);
  const PagedSeq s = paged_seq(a.batch, seq, a.status);
  if (rt * kRows >= s.n * a.G) return;
  const RowTile g = row_tile(a, s, rt);
  if (g.active <= 1) return;  // written by the split itself
  const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * kCols;
  if (g.r0 + row >= g.rows) return;
  const float* pl = a.part_lse + item * a.splits * kRows + row;
  const float* po = a.part_o + (item * a.splits * kRows + row) * D + c0;
  float m = -INFINITY;
  for (int i = 0; i < g.active; ++i) m = fmaxf(m, pl[i * kRows]);
  const float mu = m == -INFINITY ? 0.f : m;
  float sum = 0.f, x[kCols] = {};
  for (int i = 0; i < g.active; ++i) {
    const float w = ex2(pl[i * kRows] - mu);
    sum += w;
    const float* src = po + static_cast<long long>(i) * kRows * D;
#pragma unroll
    for (int c = 0; c < kCols; c += 4) {
      const float4 v = *reinterpret_cast<const float4*>(src + c);
      x[c] = fmaf(w, v.x, x[c]);
      x[c + 1] = fmaf(w, v.y, x[c + 1]);
      x[c + 2] = fmaf(w, v.z, x[c + 2]);
      x[c + 3] = fmaf(w, v.w, x[c + 3]);
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kCols; ++i) x[i] *= f;
  const long long at = static_cast<long long>(s.row0 + (g.r0 + row) / a.G) * a.Hq + h * a.G + (g.r0 + row) % a.G;
  uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + c0);
#pragma unroll
  for (int i = 0; i < kCols; i += 8)
    dst[i / 8] = make_uint4(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]),
                            pack_bf16(x[i + 4], x[i + 5]), pack_bf16(x[i + 6], x[i + 7]));
  if (c0 == 0) a.lse[at] = sum == 0.f ? -INFINITY : kLn2 * (m + log2f(sum));
}

template <int D>
int launch_rows(const PagedPool& pool, const AttnArgs& a, long long items, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap mk, mv;
  const int box = pool.page_size < kTile ? pool.page_size : kTile;
  const int blocks = pool.num_pages * pool.num_heads;
  if (!make_map_pages(&mk, pool.k_pages, blocks, pool.page_size, D, box) ||
      !make_map_pages(&mv, pool.v_pages, blocks, pool.page_size, D, box))
    return -3;
  const bool half = a.batch.max_q * a.G <= 8;
  auto kern = half ? paged_rows_kernel<D, true> : paged_rows_kernel<D, false>;
  // attribute slots 20 to 23
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, 20 + (D == 128 ? 2 : 0) + (half ? 1 : 0)))
    return -3;
  const long long grid = items * a.splits;
  if (grid > 0x7fffffffLL) return -1;
  cudaError_t e = launch_overlapped(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), C::kSmemBytes,
                                    stream, mk, mv, a);
  if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) return -3;
  if (a.splits > 1) {
    e = launch_overlapped(paged_merge_kernel<D>, dim3(static_cast<unsigned>(items)), dim3(128), 0, stream, a);
    if (cudaGetLastError() != cudaSuccess || e != cudaSuccess) return -3;
  }
  return 0;
}

}  // namespace

PagedSplit paged_attn_split(const PagedPool& pool, const PagedBatchDev& batch, int Hq, int max_kv,
                            int n_splits, int sms) {
  PagedSplit r{};
  const int G = Hq / pool.num_heads;
  r.row_tiles = static_cast<int>((static_cast<long long>(batch.max_q) * G + kRows - 1) / kRows);
  const long long items = static_cast<long long>(batch.B) * pool.num_heads * r.row_tiles;
  const long long tiles = max_kv > 0 ? (static_cast<long long>(max_kv) + kTile - 1) / kTile : 1;
  long long per = tiles;  // tiles per split
  if (n_splits > 0) {
    per = (tiles + n_splits - 1) / n_splits;
  } else {
    const long long slots = 2LL * sms;
    const long long total = items * tiles;
    per = total <= slots ? 1 : total < 8 * slots ? (total + slots - 1) / slots
                                                 : (total + 3 * slots - 1) / (3 * slots);
    if (total >= 8 * slots && per < 8) per = 8;
    if (per > tiles) per = tiles;
  }
  r.split_tiles = static_cast<int>(per);
  r.splits = static_cast<int>((tiles + per - 1) / per);
  r.workspace_bytes =
      r.splits > 1 ? static_cast<size_t>(items) * r.splits * kRows * (pool.d + 1) * sizeof(float) : 0;
  return r;
}

int launch_paged_attn(const PagedPool& pool, const PagedBatchDev& batch, const PagedAttn& p,
                      const PagedSplit& split, void* workspace, cudaStream_t stream) {
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
  a.G = p.Hq / pool.num_heads;
  a.window = p.window;
  a.row_tiles = split.row_tiles;
  a.splits = split.splits;
  a.split_tiles = split.split_tiles;
  // scale 0 (uniform weights) runs as a tiny positive scale, as in the forward
  const float sl2 = p.scale * kLog2e;
  a.scale_log2 = sl2 > 1e-30f ? sl2 : 1e-30f;
  const long long items = static_cast<long long>(batch.B) * pool.num_heads * split.row_tiles;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (split.splits > 1 ? items * split.splits * kRows * pool.d : 0);
  return pool.d == 64 ? launch_rows<64>(pool, a, items, stream) : launch_rows<128>(pool, a, items, stream);
}

}  // namespace fa
