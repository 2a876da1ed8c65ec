// qmv_gate.hip -- routing to experts by softmax or sigmoid scores, a bias,
// groups and renormalised weights, for gfx950.
//
// Which expert is chosen is decided at a border, so everything up to the choice
// is held in fp64: fp32 logits of another summing order would pick others
// where two choices are within 1e-7 of each other, and the routed matvecs of
// two steps over the same token would differ.
#include "qmv_device.h"
#include "qmv_steps.h"

namespace qmv {

namespace {

constexpr int kGateWaves = 8;
constexpr int kGatePer = 16;  // experts of a lane at most

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp_i<CTRL>((int)(uint32_t)(b >> 32));
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ double lane_d(double v, int lane) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

// Sum and largest over the wave, in every lane alike.
__device__ __forceinline__ double wave_sum_d(double v) {
  v += dpp_d<DPP_XOR1>(v);
  v += dpp_d<DPP_XOR2>(v);
  v += dpp_d<DPP_HALF_MIRROR>(v);
  v += dpp_d<DPP_MIRROR>(v);
  return (lane_d(v, 0) + lane_d(v, 16)) + (lane_d(v, 32) + lane_d(v, 48));
}
__device__ __forceinline__ double wave_max_d(double v) {
  v = fmax(v, dpp_d<DPP_XOR1>(v));
  v = fmax(v, dpp_d<DPP_XOR2>(v));
  v = fmax(v, dpp_d<DPP_HALF_MIRROR>(v));
  v = fmax(v, dpp_d<DPP_MIRROR>(v));
  return fmax(fmax(lane_d(v, 0), lane_d(v, 16)), fmax(lane_d(v, 32), lane_d(v, 48)));
}
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<DPP_XOR1>((int)v));
  v = max(v, (uint32_t)dpp_i<DPP_XOR2>((int)v));
  v = max(v, (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)v));
  v = max(v, (uint32_t)dpp_i<DPP_MIRROR>((int)v));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// A double's place in the order, as an unsigned number: above 0 for every
// value; NaN counts as -inf, and -0 as +0.
__device__ __forceinline__ uint64_t place(double v) {
  if (!(v == v)) v = -__builtin_inf();
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// The lane that holds the largest key of the wave, the lowest index among
// equal ones; key 0: none.  In every lane alike.
__device__ __forceinline__ int wave_first(uint64_t key, int index) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const uint32_t mh = wave_max_u(hi);
  uint64_t b = __ballot(hi == mh);
  if (__popcll(b) > 1) {
    const uint32_t ml = wave_max_u(hi == mh ? lo : 0u);
    b = __ballot(hi == mh && lo == ml);
    if (__popcll(b) > 1) {
      const uint32_t mi = wave_max_u(hi == mh && lo == ml ? ~(uint32_t)index : 0u);
      b = __ballot(hi == mh && lo == ml && ~(uint32_t)index == mi);
    }
  }
  return __ffsll((unsigned long long)b) - 1;
}

// One token's choice by one wave.  l: the lane's logits, of experts lane + 64 i;
// sc: an array of n_experts doubles in LDS of this wave's own.
__device__ __forceinline__ void gate_select(const GateArgs& a, int t, double (&l)[kGatePer], double* sc) {
  const int lane = threadIdx.x & 63;
  const int per = (a.n_experts + 63) / 64;
  // scores
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (i < per) l[i] = 1.0 / (1.0 + exp(-l[i]));
  } else {
    double m = -__builtin_inf(), sum = 0.0;
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (lane + 64 * i < a.n_experts) m = fmax(m, l[i]);
    m = wave_max_d(m);
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (i < per) {
        l[i] = exp(l[i] - m);
        if (lane + 64 * i < a.n_experts) sum += l[i];
      }
    sum = wave_sum_d(sum);
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (i < per) l[i] = l[i] / sum;
  }
  // choices: with the bias, in LDS for the groups
  double c[kGatePer];
  uint32_t in = 0;  // bit i: expert lane + 64 i may be chosen
#pragma unroll
  for (int i = 0; i < kGatePer; ++i) {
    const int e = lane + 64 * i;
    c[i] = 0.0;
    if (e < a.n_experts) {
      c[i] = l[i] + (a.bias != nullptr ? (double)a.bias[e] : 0.0);
      in |= 1u << i;
    }
  }
  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (lane + 64 * i < a.n_experts) sc[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    const int size = a.n_experts / a.groups;
    uint64_t key = 0;
    if (lane < a.groups) {  // a group's worth: its largest one or two
      double u = -__builtin_inf(), v = u;
      for (int i = 0; i < size; ++i) {
        double w = sc[lane * size + i];
        w = w == w ? w : -__builtin_inf();
        v = fmax(v, fmin(u, w));
        u = fmax(u, w);
      }
      key = place(a.group_best == 2 ? u + v : u);
    }
    uint64_t kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const int g = wave_first(key, lane);
      kept |= 1ull << g;
      if (lane == g) key = 0;
    }
#pragma unroll
    for (int i = 0; i < kGatePer; ++i) {
      const int e = lane + 64 * i;
      if (e < a.n_experts && !((kept >> (e / size)) & 1)) in &= ~(1u << i);
    }
    __builtin_amdgcn_wave_barrier();
  }
  // the largest one after the other
  uint64_t key = 0;
  int at = 0;
  auto best = [&]() {
    key = 0;
    at = 0;
#pragma unroll
    for (int i = 0; i < kGatePer; ++i)
      if (i < per && (in >> i) & 1) {
        const uint64_t p = place(c[i]);
        if (p > key) {
          key = p;
          at = i;
        }
      }
  };
  best();
  double mine = 0.0, total = 0.0;
  int id = 0;
  for (int j = 0; j < a.top_k; ++j) {
    const int w = wave_first(key, lane + 64 * at);
    double s = l[0];
#pragma unroll
    for (int i = 1; i < kGatePer; ++i) s = at == i ? l[i] : s;
    s = lane_d(s, w);
    const int e = w + 64 * __builtin_amdgcn_readlane(at, w);
    total += s;
    if (lane == j) {
      id = e;
      mine = s;
    }
    if (lane == w) {
      in &= ~(1u << at);
      best();
    }
  }
  if (lane < a.top_k) {
    double w = mine;
    if (a.renorm) w = total == 0.0 ? 1.0 / a.top_k : mine / total;
    a.ids[(int64_t)t * a.top_k + lane] = id;
    a.weights[(int64_t)t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

// EG experts x TG tokens x 4 columns of a lane.
template <int EG, int TG>
struct GateChunk {
  f32x4 w[EG];
  f32x4 x[TG];
  __device__ __forceinline__ void load(const GateArgs& a, int e0, int t0, int c) {
#pragma unroll
    for (int e = 0; e < EG; ++e)
      w[e] = *reinterpret_cast<const f32x4*>(a.wr + (int64_t)min(e0 + e, a.n_experts - 1) * a.k + c);
#pragma unroll
    for (int t = 0; t < TG; ++t)
      x[t] = *reinterpret_cast<const f32x4*>(a.x + (int64_t)min(t0 + t, a.n_tok - 1) * a.ldx + c);
  }
  __device__ __forceinline__ void fma_into(double (&acc)[EG * TG]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double wd[EG], xd[TG];
#pragma unroll
      for (int e = 0; e < EG; ++e) wd[e] = (double)w[e][i];
#pragma unroll
      for (int t = 0; t < TG; ++t) xd[t] = (double)x[t][i];
#pragma unroll
      for (int e = 0; e < EG; ++e)
#pragma unroll
        for (int t = 0; t < TG; ++t) acc[e * TG + t] = fma(wd[e], xd[t], acc[e * TG + t]);
    }
  }
};

}  // namespace

// l[t][e] = sum over c of wr[e][c] x[t][c] in fp64 (products of fp32 numbers
// are exact there), EG experts by TG tokens a workgroup whose waves share the
// columns.  Workgroups of the first experts also write the Q8 blocks of x.
template <int EG, int TG>
__global__ __launch_bounds__(64 * kGateWaves) void k_gate_logits(GateArgs a) {
  constexpr int P = EG * TG;
  __shared__ double red[kGateWaves][P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = blockIdx.x * EG, t0 = blockIdx.y * TG;
  double acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.0;
  constexpr int kStep = 4 * 64 * kGateWaves;
  const bool qx = a.qs != nullptr && blockIdx.x == 0;
  auto put = [&](const GateChunk<EG, TG>& ch, int col) {
#pragma unroll
    for (int t = 0; t < TG; ++t) {
      if (t0 + t < a.n_tok) {  // uniform
        const float vv[4] = {ch.x[t].x, ch.x[t].y, ch.x[t].z, ch.x[t].w};
        float db;
        int sum;
        const uint32_t packed = q8_block8(vv, db, sum);
        *reinterpret_cast<uint32_t*>(a.qs + (int64_t)(t0 + t) * a.k + col) = packed;
        if ((lane & 7) == 0) {
          a.qd[(int64_t)(t0 + t) * (a.k / 32) + col / 32] = db;
          a.qsum[(int64_t)(t0 + t) * (a.k / 32) + col / 32] = sum;
        }
      }
    }
  };
  for (int c = 4 * (lane + 64 * wave); c < a.k; c += kStep) {
    GateChunk<EG, TG> ch;
    ch.load(a, e0, t0, c);
    if (qx) put(ch, c);
    ch.fma_into(acc);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double v = wave_sum_d(acc[i]);
    if (lane == 0) red[wave][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < P) {
    double s = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kGateWaves; ++w) s += red[w][threadIdx.x];
    const int e = e0 + threadIdx.x / TG, t = t0 + threadIdx.x % TG;
    if (e < a.n_experts && t < a.n_tok) a.logits[(int64_t)t * a.n_experts + e] = s;
  }
}

// One wave a token.
__global__ __launch_bounds__(64) void k_gate_select(GateArgs a) {
  __shared__ double sc[64 * kGatePer];
  const int t = blockIdx.x, lane = threadIdx.x;
  double l[kGatePer];
#pragma unroll
  for (int i = 0; i < kGatePer; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < a.n_experts ? a.logits[(int64_t)t * a.n_experts + e] : 0.0;
    if (a.logits_out != nullptr && e < a.n_experts) a.logits_out[(int64_t)t * a.n_experts + e] = (float)l[i];
  }
  gate_select(a, t, l, sc);
}

namespace {

template <int EG, int TG>
void launch_logits(const GateArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.n_experts + EG - 1) / EG), (unsigned)((a.n_tok + TG - 1) / TG));
  hipLaunchKernelGGL((k_gate_logits<EG, TG>), grid, dim3(64 * kGateWaves), 0, st, a);
}

}  // namespace

hipError_t launch_router_gate(const GateArgs& a, hipStream_t st) {
  if (a.n_tok == 1) launch_logits<1, 1>(a, st);
  else if (a.n_tok == 2) launch_logits<2, 2>(a, st);
  else launch_logits<4, 4>(a, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_gate_select, dim3((unsigned)a.n_tok), dim3(64), 0, st, a);
  return hipGetLastError();
}

}  // namespace qmv
