// Rotary positions with several axes: queries and keys of packed rows.
//
// Mathematics. Channel pair i of the first `rot` channels of a head turns by
// the angle of the token's position on the pair's own axis: with p =
// positions[axis_of[i]][t],
//   (a, b) -> (a cos[p, i] - b sin[p, i], b cos[p, i] + a sin[p, i]),
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved. The map is
// orthogonal, so its gradient is the rotation by the negative angle (inverse).
// Products and sums are rounded one by one in fp32, as in fa_paged_append.cu,
// so a query turned here has the bits of one turned there.
//
// What bounds it: memory. Per token 4 d bytes for each head (read and write)
// and 4 rot of the tables, which the tokens of a picture share in L2. A thread
// keeps the angles of 16 channels (8 pairs) in registers and takes them
// through up to kHeads heads of its token, whose loads are all in flight at once;
// eight neighbouring threads cover 128-byte lines.
// Measured: 32768 tokens, 32 + 8 heads, d = 128, three axes: 104.6 us, 97 % of the
// rate of a plain copy; 10007 tokens, 16 + 16 heads, d = 64, interleaved: 16.5 us one
// call after another, 75 % (a launch of 16 us ends before its loads run at full rate
// for long), 12.6 as replays of a graph, whose 85 MB stay in L2.

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads whose loads a thread has in flight

struct RopeArgs {
  const __nv_bfloat16* x[2];  // queries, keys
  __nv_bfloat16* y[2];
  long long x_stride[2], y_stride[2];
  const int* positions;
  const float* cos;
  const float* sin;
  int* status;
  int H, Hq;           // heads of both, and of the queries
  int T, rot, max_pos;
  int interleaved, inverse;
  int slots, tokens;   // threads' places per token for heads, and tokens per block
  RopeAxes axes;
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const RopeArgs a) {
  constexpr int kUnits = D / 16;
  grid_dep_wait();
  grid_dep_launch();
  const int unit = threadIdx.x % kUnits, place = threadIdx.x / kUnits;
  const int tl = place / a.slots, slot = place - tl * a.slots;
  const long long t = static_cast<long long>(blockIdx.x) * a.tokens + tl;
  if (tl >= a.tokens || t >= a.T) return;

  // this thread's two runs of eight channels, and its pairs' column in the tables
  const bool turns = unit * 16 < a.rot;
  const bool halves = turns && !a.interleaved;
  const int c0 = halves ? unit * 8 : unit * 16, c1 = halves ? c0 + a.rot / 2 : c0 + 8, col = unit * 8;
  float c[8], s[8];
  bool have = false;
  for (int h0 = slot; h0 < a.H; h0 += kHeads * a.slots) {
    uint4 w[kHeads][2];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * a.slots;
      if (h >= a.H) continue;
      const int k = h >= a.Hq ? 1 : 0;
      const __nv_bfloat16* row = a.x[k] + t * a.x_stride[k] + static_cast<long long>(h - k * a.Hq) * D;
      w[i][0] = *reinterpret_cast<const uint4*>(row + c0);
      w[i][1] = *reinterpret_cast<const uint4*>(row + c1);
    }
    if (turns && !have) {
      have = true;
      bool bad = false;
      auto position = [&](int i) {
        const int p = __ldg(a.positions + static_cast<long long>(a.axes.of[i]) * a.T + t);
        bad = bad || p < 0 || p >= a.max_pos;
        return min(max(p, 0), a.max_pos - 1);
      };
      const long long half = a.rot / 2;
      if (a.axes.whole >> unit & 1) {  // the eight pairs are on one axis
        const long long at = position(col) * half + col;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos + at + i));
          const float4 y = __ldg(reinterpret_cast<const float4*>(a.sin + at + i));
          c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
          s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const long long at = position(col + i) * half + col + i;
          c[i] = __ldg(a.cos + at);
          s[i] = __ldg(a.sin + at);
        }
      }
      if (bad) raise_index(a.status);
      if (a.inverse) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * a.slots;
      if (h >= a.H) continue;
      const int k = h >= a.Hq ? 1 : 0;
      __nv_bfloat16* row = a.y[k] + t * a.y_stride[k] + static_cast<long long>(h - k * a.Hq) * D;
      if (turns) {
        float x[16];
        unpack8(w[i][0], x);
        unpack8(w[i][1], x + 8);
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(x[2 * j], x[2 * j + 1], c[j], s[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(x[j], x[j + 8], c[j], s[j]);
        }
        w[i][0] = pack8(x);
        w[i][1] = pack8(x + 8);
      }
      *reinterpret_cast<uint4*>(row + c0) = w[i][0];
      *reinterpret_cast<uint4*>(row + c1) = w[i][1];
    }
  }
}

}  // namespace

int launch_rope_axes(const RopeProblem& p, cudaStream_t stream) {
  RopeArgs a{};
  const int H = p.Hq + p.Hk, units = p.d / 16;
  a.x[0] = static_cast<const __nv_bfloat16*>(p.q);
  a.x[1] = static_cast<const __nv_bfloat16*>(p.k);
  a.y[0] = static_cast<__nv_bfloat16*>(p.q_out);
  a.y[1] = static_cast<__nv_bfloat16*>(p.k_out);
  a.x_stride[0] = p.q_stride;
  a.x_stride[1] = p.k_stride;
  a.y_stride[0] = p.q_out_stride;
  a.y_stride[1] = p.k_out_stride;
  a.positions = p.positions;
  a.cos = p.cos;
  a.sin = p.sin;
  a.status = device_status_word();
  a.H = H;
  a.Hq = p.Hq;
  a.T = p.T;
  a.rot = p.rot;
  a.max_pos = p.max_pos;
  a.interleaved = p.interleaved;
  a.inverse = p.inverse;
  a.axes = p.axes;
  const int sms = device_sm_count();
  if (!a.status || sms <= 0) return -3;
  // Few tokens: a thread per head. Many: kHeads heads per thread.
  const bool few = static_cast<long long>(p.T) * H * units <= static_cast<long long>(sms) * kThreads * 2;
  const int most = kThreads / units, want = few ? H : (H + kHeads - 1) / kHeads;
  a.slots = want < most ? want : most;
  a.tokens = most / a.slots;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.T) + a.tokens - 1) / a.tokens);
  auto kern = p.d == 64 ? rope_axes_kernel<64> : p.d == 128 ? rope_axes_kernel<128> : rope_axes_kernel<256>;
  const cudaError_t e = launch_overlapped(kern, dim3(grid), dim3(kThreads), 0, stream, a);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace fa
