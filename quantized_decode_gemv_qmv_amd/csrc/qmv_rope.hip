// qmv_rope.hip -- root-mean-square norm of each query and key head and its
// rotation by the token's positions, one pass, for gfx950.
#include "qmv_device.h"
#include "qmv_steps.h"

namespace qmv {

namespace {

constexpr int kHeadWaves = 4;  // of a workgroup
constexpr int kHeadBatch = 4;  // vectors of a lane whose loads are in flight together, about

// cos and sin of pos * freq.  The product of a 31-bit and a 24-bit number and
// its turns (times 1 / 2 pi, which two doubles hold to 107 bits) keep their low
// parts, so the place in the circle is right to 2^-45 turns at every position;
// the angle's rest within +-pi/4 is rounded to fp32 once and the Taylor sums
// end below 2^-28 there.
__device__ __forceinline__ void cos_sin(int pos, float freq, float& c, float& s) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3;      // 1 / (2 pi)
  constexpr double kTurnLow = -0x1.6b01ec5417056p-57;  // what kTurn leaves of it
  const double p = (double)pos, f = (double)freq;
  const double a = p * f;
  const double whole = rint(a * kTurn);
  const double low = fma(a, kTurnLow, fma(p, f, -a) * kTurn);
  const double part = fma(a, kTurn, -whole) + low;  // turns, within +-1/2 where a is below 2^53 of them
  const double quarter = rint(4.0 * part);
  const float z = (float)(fma(-0.25, quarter, part) * 6.283185307179586477);
  const float z2 = z * z;
  // Taylor sums, up to z^9 / 9! and z^10 / 10!
  float sn = fmaf(z2, 2.75573192e-6f, -1.98412698e-4f);
  sn = fmaf(z2, sn, 8.33333333e-3f);
  sn = fmaf(z2, sn, -0.166666667f);
  sn = fmaf(z * z2, sn, z);
  float cs = fmaf(z2, -2.75573192e-7f, 2.48015873e-5f);
  cs = fmaf(z2, cs, -1.38888889e-3f);
  cs = fmaf(z2, cs, 4.16666667e-2f);
  cs = fmaf(z2, cs, -0.5f);
  cs = fmaf(z2, cs, 1.0f);
  const int q = (int)quarter & 3;  // -2 .. 2
  const float u = (q & 1) ? sn : cs, v = (q & 1) ? cs : sn;
  c = (q == 1 || q == 2) ? -u : u;
  s = (q & 2) ? -v : v;
}

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp_i<CTRL>((int)(uint32_t)(b >> 32));
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

// Sum over each aligned group of L lanes (4 .. 64), in every lane of it.
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
  v += dpp_d<DPP_XOR1>(v);
  v += dpp_d<DPP_XOR2>(v);
  if constexpr (L >= 8) v += dpp_d<DPP_HALF_MIRROR>(v);
  if constexpr (L >= 16) v += dpp_d<DPP_MIRROR>(v);
  if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
  if constexpr (L >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

}  // namespace

// y = turn(x * inv * w): a wave takes 64 / L heads of one token a pass, L lanes
// a head with four dims each (or V times four), and a lane has the same dims in
// every pass.  Cosines and sines are made once a wave, one or two pairs a lane, and
// come to the dims' lanes through LDS (each lane its own dims': 8192 x 72 132 -> 122
// us).  Squares are summed in fp64 (each is exact, no length of x overflows it).  A
// pair's other half lies in the lane (neighbouring pairs) or comes through LDS.  One
// read and one write of every value bound it: 8192 tokens x 72 heads of 128 dims 106
// us, 5.7 TB/s (a large copy reaches 4.9); one token 3.1 us, the launch and two loads
// in a row.  All loads of a wave's first passes are on their way before its angles
// are made.
// V4: the halves' distance is a multiple of four dims, so the partner values
// of a lane are one 16-byte vector.  NT: stores that pass the caches by.
// V: vectors of a lane, 4 L dims apart.
template <int L, int V, bool ADJACENT, bool V4, bool NT>
__global__ __launch_bounds__(64 * kHeadWaves) void k_head_norm_rope(HeadsArgs a) {
  constexpr int HPP = 64 / L;         // heads of a pass
  constexpr int kHead = 4 * L * V;    // room of a head
  constexpr int kBatch = V == 1 ? kHeadBatch : kHeadBatch / 2;
  constexpr int kPairs = kHead > 128 ? 2 : 1;  // of a lane
  __shared__ __align__(16) float s_x[kHeadWaves][256 * V];
  __shared__ float s_cos[kHeadWaves][64 * kPairs], s_sin[kHeadWaves][64 * kPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t g = (int64_t)blockIdx.x * kHeadWaves + wave;
  const int t = (int)(g / a.waves_a_token), part = (int)(g % a.waves_a_token);
  if (t >= a.n_tok) return;  // no barrier below
  const int d0 = 4 * (lane % L);
  const int total = a.heads[0] + a.heads[1];
  // the token's rows (a head lies below 2^23 values in its row)
  const float *xq = a.x[0] + t * a.ldx[0], *xk = a.x[1] + t * a.ldx[1];
  float *yq = a.y[0] + t * a.ldy[0], *yk = a.y[1] + t * a.ldy[1];
  // a pass's values; the next ones are on their way while a batch is worked on
  auto fetch = [&](int p, f32x4 (&x)[V]) {
    const int h = p * HPP + lane / L;
    const int m = h >= a.heads[0];
    const float* from = (m ? xk : xq) + (h - (m ? a.heads[0] : 0)) * a.dim;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = d0 + 4 * L * v;
      x[v] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (p < a.passes && h < total && d < a.dim) x[v] = *reinterpret_cast<const f32x4*>(from + d);
    }
  };
  f32x4 x[kBatch][V];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) fetch(part + b * a.waves_a_token, x[b]);
  f32x4 wq[V], wk[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int d = d0 + 4 * L * v;
    wq[v] = wk[v] = f32x4{1.f, 1.f, 1.f, 1.f};
    if (a.w[0] != nullptr && d < a.dim) wq[v] = *reinterpret_cast<const f32x4*>(a.w[0] + d);
    if (a.w[1] != nullptr && d < a.dim) wk[v] = *reinterpret_cast<const f32x4*>(a.w[1] + d);
  }
  // cosines and sines of the pairs, one or two a lane, which all heads share
  const int half = a.rot / 2;
  const int first_pos = a.pos != nullptr ? a.pos[t] : 0;
  float freq[kPairs];
  int axis[kPairs];
#pragma unroll
  for (int n = 0; n < kPairs; ++n) {
    const int i = lane + 64 * n;
    freq[n] = 0.f;
    axis[n] = -1;
    if (i < half) {
      freq[n] = a.freq[i];
      axis[n] = a.axis != nullptr ? a.axis[i] : 0;
      if (axis[n] >= a.n_axes) axis[n] = -1;
    }
  }
  if (first_pos < 0) return;
  uint64_t turns[kPairs];  // pairs that turn
#pragma unroll
  for (int n = 0; n < kPairs; ++n) {
    turns[n] = __ballot(axis[n] >= 0);
    if (axis[n] >= 0) {
      const int pos = axis[n] == 0 ? first_pos : a.pos[(int64_t)axis[n] * a.n_tok + t];
      float c, s;
      cos_sin(pos, freq[n], c, s);
      s_cos[wave][lane + 64 * n] = c * a.scale;
      s_sin[wave][lane + 64 * n] = s * a.scale;
    }
  }
  __builtin_amdgcn_wave_barrier();
  // those of the lane's dims
  float c[V][4], s[V][4];
  int other[V][4];
  bool turn[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = d0 + 4 * L * v + j;
      const bool second = ADJACENT ? j & 1 : d >= half;
      const int i = ADJACENT ? d >> 1 : (second ? d - half : d);
      other[v][j] = d;
      turn[v][j] = false;
      c[v][j] = s[v][j] = 0.f;
      if (d < a.rot) {
        if (!ADJACENT) other[v][j] = second ? i : d + half;
        turn[v][j] = (turns[kPairs == 2 ? i >> 6 : 0] >> (i & 63)) & 1;
        c[v][j] = s_cos[wave][i];
        s[v][j] = second ? s_sin[wave][i] : -s_sin[wave][i];
      }
    }
  float* sx = s_x[wave] + lane / L * kHead;  // the head's values
  for (int p0 = part; p0 < a.passes; p0 += a.waves_a_token * kBatch) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int p = p0 + b * a.waves_a_token;
      if (p >= a.passes) break;  // uniform
      const int h = p * HPP + lane / L;
      const int m = h >= a.heads[0];
      f32x4 y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = x[b][v];
      fetch(p + kBatch * a.waves_a_token, x[b]);
      double ss = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) ss += (double)y[v][j] * (double)y[v][j];
      ss = lanes_sum<L>(ss);
      if (m ? a.w[1] != nullptr : a.w[0] != nullptr) {
        // 1 / sqrt: the hardware's, right to 2^-24, and a Newton step
        const double ms = fma(ss, a.inv_dim, a.eps);
        double inv = __builtin_amdgcn_rsq(ms);
        inv *= fma(-0.5 * ms * inv, inv, 1.5);
        // fp32 holds it below its normal numbers: 2^64 from the values to it; and
        // with an infinity in the head it is 0, where the step made no number
        if (__builtin_expect(__any(ms > 0x1p250), 0)) {
          const bool far = ms > 0x1p250;
          if (far) inv = ms < __builtin_inf() ? inv * 0x1p64 : 0.0;
#pragma unroll
          for (int v = 0; v < V; ++v) y[v] *= far ? 0x1p-64f : 1.f;
        }
        const float r = (float)inv;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) y[v][j] = (y[v][j] * r) * (m ? wk[v][j] : wq[v][j]);
      }
      f32x4 q[V];
      if constexpr (ADJACENT) {
#pragma unroll
        for (int v = 0; v < V; ++v) q[v] = f32x4{y[v][1], y[v][0], y[v][3], y[v][2]};
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) *reinterpret_cast<f32x4*>(sx + d0 + 4 * L * v) = y[v];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if constexpr (V4) {
            q[v] = *reinterpret_cast<const f32x4*>(sx + other[v][0]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[v][j] = sx[other[v][j]];
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
      float* to = (m ? yk : yq) + (h - (m ? a.heads[0] : 0)) * a.dim;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int d = d0 + 4 * L * v;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[v][j] = turn[v][j] ? fmaf(y[v][j], c[v][j], q[v][j] * s[v][j]) : y[v][j];
        if (h < total && d < a.dim) {
          if constexpr (NT)
            __builtin_nontemporal_store(y[v], reinterpret_cast<f32x4*>(to + d));
          else
            *reinterpret_cast<f32x4*>(to + d) = y[v];
        }
      }
    }
  }
}

namespace {

template <int L, int V, bool ADJACENT, bool V4>
hipError_t launch(const HeadsArgs& a, unsigned grid, bool stream, hipStream_t st) {
  const dim3 b(64 * kHeadWaves);
  if constexpr (V == 1) {
    if (!stream) {
      hipLaunchKernelGGL((k_head_norm_rope<L, V, ADJACENT, V4, false>), dim3(grid), b, 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_head_norm_rope<L, V, ADJACENT, V4, true>), dim3(grid), b, 0, st, a);
  return hipGetLastError();
}

// Outputs that the caches would not keep for the next step pass them by (10 MB
// 9.6 -> 8.6 us, 20 MB 16.6 -> 11.6, 302 MB 136 -> 130).
bool streams(const HeadsArgs& a) {
  return (int64_t)a.n_tok * (a.heads[0] + a.heads[1]) * a.dim * 4 > (int64_t(8) << 20);
}

template <int L, int V>
hipError_t launch(HeadsArgs a, int cus, hipStream_t st) {
  const int total = a.heads[0] + a.heads[1], hpp = 64 / L;
  a.passes = (total + hpp - 1) / hpp;
  // a wave a pass until a compute unit has eight, then up to eight passes a wave (of
  // three vectors, up to three), which share the angles
  int64_t per = (int64_t)a.n_tok * a.passes / ((int64_t)cus * 8);
  const int64_t most = V == 1 ? 8 : 3;
  per = per < 1 ? 1 : (per > most ? most : per);
  // below 2^25 waves, which is 2^31 threads (65536 tokens have 65536 at least)
  const int64_t least = ((int64_t)a.n_tok * a.passes >> 24) + 1;
  if (per < least) per = least;
  a.waves_a_token = (int)((a.passes + per - 1) / per);
  const int64_t waves = (int64_t)a.n_tok * a.waves_a_token;
  const unsigned grid = (unsigned)((waves + kHeadWaves - 1) / kHeadWaves);
  const bool stream = streams(a);
  if (a.adjacent) return launch<L, V, true, true>(a, grid, stream, st);
  if (a.rot % 8 == 0) return launch<L, V, false, true>(a, grid, stream, st);
  return launch<L, V, false, false>(a, grid, stream, st);
}

// L lanes a head of more than 2 L dims, or, in large calls where that takes fewer
// vectors in all, L / 4 lanes of three vectors each: heads of 96 dims leave no lane
// idle then (6237 x 48 heads of 96 61 -> 46 us, 5877 x 24 of 192 58 -> 42).
template <int L>
hipError_t launch_wide(const HeadsArgs& a, int cus, hipStream_t st) {
  const int total = a.heads[0] + a.heads[1], one = 64 / L, three = 4 * one;
  if (a.dim <= 3 * L && streams(a) && 3 * ((total + three - 1) / three) < (total + one - 1) / one)
    return launch<L / 4, 3>(a, cus, st);
  return launch<L, 1>(a, cus, st);
}

}  // namespace

hipError_t launch_head_norm_rope(const HeadsArgs& a, int cus, hipStream_t st) {
  if (a.dim <= 16) return launch<4, 1>(a, cus, st);
  if (a.dim <= 32) return launch<8, 1>(a, cus, st);
  if (a.dim <= 64) return launch_wide<16>(a, cus, st);
  if (a.dim <= 128) return launch_wide<32>(a, cus, st);
  return launch_wide<64>(a, cus, st);
}

}  // namespace qmv
