// qmv_gate.hip -- routing to experts by softmax or sigmoid scores, a bias,
// groups and renormalised weights, for gfx950.
//
// Which expert is chosen is decided at a border, so everything up to the choice
// is held in fp64: fp32 logits of another summing order would pick others
// where two choices are within 1e-7 of each other, and the routed matvecs of
// two steps over the same token would differ.
//
// Up to four tokens one launch does it all (1 x 128 experts of 4096 columns 6.3 us:
// the launch, one load of the weights, the handoff to the last workgroup of some 2
// us, its choice of some 2); more tokens take the matrix unit and a second launch
// (64 x 256 of 5120: 14.5 us, of which 8.7 and 6.6; the products alone would take
// 2.1).  On the vector ALU the logits of 64 tokens took 15.4 us; chosen by the last
// workgroup of 16 tokens, 64 tokens took 18 to 26 us in one launch.
#include "qmv_device.h"
#include "qmv_steps.h"

namespace qmv {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kGateWaves = 16;
constexpr int kGateTile = 16;  // experts and tokens of a matrix product
// Steps whose loads are in flight (3 / 5 / 8: 16 x 128 of 4096 8.6 / 8.6 / 8.7 us, 64 x 256
// of 5120 13.0 / 13.2 / 13.1, of 7168 14.9 / 15.1 / 14.9, 64 x 384 of 7168 22.5 / 23.2 / 24.0).
constexpr int kGateAhead = 5;
constexpr int kFewExperts = 4; // of a workgroup, up to four tokens

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

// One token's choice by one wave.  l and bias: the lane's logits and biases, of
// experts lane + 64 i; sc: an array of 64 PER doubles in LDS of this wave's own.
template <int PER>
__device__ __forceinline__ void gate_select(const GateArgs& a, int t, double (&l)[PER], const float (&bias)[PER], double* sc) {
  const int lane = threadIdx.x & 63;
  // scores
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = 1.0 / (1.0 + exp(-l[i]));
  } else {
    double m = -__builtin_inf(), sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < a.n_experts) m = fmax(m, l[i]);
    m = wave_max_d(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = exp(l[i] - m);
      if (lane + 64 * i < a.n_experts) sum += l[i];
    }
    const double inv = 1.0 / wave_sum_d(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] *= inv;
  }
  // choices: with the bias; 0 is below each of them
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0;
    if (e < a.n_experts) {
      const double c = l[i] + (double)bias[i];
      key[i] = place(c);
      if (a.groups > 1) sc[e] = c;
    }
  }
  if (a.groups > 1) {
    __builtin_amdgcn_wave_barrier();
    const int size = a.n_experts / a.groups;
    // a group's worth, its largest one or two: S lanes a group
    int shift = 6;
    while ((a.groups << shift) > 64) --shift;
    const int g = lane >> shift, first = lane & ((1 << shift) - 1);
    double u = -__builtin_inf(), v = u;
    if (g < a.groups) {
      for (int i = first; i < size; i += 1 << shift) {
        double w = sc[g * size + i];
        w = w == w ? w : -__builtin_inf();
        v = fmax(v, fmin(u, w));
        u = fmax(u, w);
      }
    }
    for (int o = 1; o < 1 << shift; o <<= 1) {
      const double p = __shfl_xor(u, o), q = __shfl_xor(v, o);
      v = fmax(fmin(u, p), fmax(v, q));
      u = fmax(u, p);
    }
    const uint64_t worth = g < a.groups ? place(a.group_best == 2 ? u + v : u) : 0;
    // a group stays if few enough are ahead of it
    int before = 0;
    for (int j = 0; j < a.groups; ++j) {
      const uint64_t other =
          ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(worth >> 32), j << shift) << 32) |
          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)worth, j << shift);
      before += other > worth || (other == worth && j < g) ? 1 : 0;
    }
    const uint64_t kept = __ballot(g < a.groups && before < a.top_groups);
    const float inv = 1.f / (float)size;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      const int of = (int)(((float)e + 0.5f) * inv);  // e / size: 0.5 / 1024 from a whole number, fp32 is off by 2^-13
      if (e < a.n_experts && !((kept >> (of << shift)) & 1)) key[i] = 0;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // the largest of the wave one after the other
  double mine = 0.0, total = 0.0;
  int id = 0;
  int at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) at[i] = i;
  if constexpr (PER <= 4) {  // each lane's in order first, so that only its head stands for it
    auto order = [&](int p, int q) {
      if (key[q] > key[p] || (key[q] == key[p] && at[q] < at[p])) {
        const uint64_t k = key[p];
        const double v = l[p];
        const int n = at[p];
        key[p] = key[q];
        l[p] = l[q];
        at[p] = at[q];
        key[q] = k;
        l[q] = v;
        at[q] = n;
      }
    };
    if constexpr (PER == 2) order(0, 1);
    if constexpr (PER == 4) {
      order(0, 1);
      order(2, 3);
      order(0, 2);
      order(1, 3);
      order(1, 2);
    }
  }
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = key[0];
    double s = l[0];
    int b = at[0];
    if constexpr (PER > 4) {
#pragma unroll
      for (int i = 1; i < PER; ++i)
        if (key[i] > best) {
          best = key[i];
          s = l[i];
          b = i;
        }
    }
    const int w = wave_first(best, lane + 64 * b);
    const int i = __builtin_amdgcn_readlane(b, w);
    s = lane_d(s, w);
    total += s;
    if (lane == j) {
      id = w + 64 * i;
      mine = s;
    }
    if (lane == w) {
      if constexpr (PER <= 4) {
#pragma unroll
        for (int q = 0; q + 1 < PER; ++q) {
          key[q] = key[q + 1];
          l[q] = l[q + 1];
          at[q] = at[q + 1];
        }
        key[PER - 1] = 0;
      } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) key[q] = q == i ? 0 : key[q];
      }
    }
  }
  if (lane < a.top_k) {
    double w = mine;
    if (a.renorm) w = total == 0.0 ? 1.0 / a.top_k : mine / total;
    a.ids[(int64_t)t * a.top_k + lane] = id;
    a.weights[(int64_t)t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

// A token's logits from the slices' sums, many loads of a lane in flight, then
// its choice.  DEVICE: the sums are another workgroup's of this launch.
template <int PER, bool DEVICE>
__device__ __forceinline__ void gate_token(const GateArgs& a, int t, double* sc) {
  constexpr int Z = PER >= 4 ? 16 / PER : 4;
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)a.n_tok * a.n_experts;
  const double* p = a.logits + (int64_t)t * a.n_experts;
  double l[PER];
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    l[i] = 0.0;
    bias[i] = a.bias != nullptr ? a.bias[min(lane + 64 * i, a.n_experts - 1)] : 0.f;
  }
  for (int z0 = 0; z0 < a.slices; z0 += Z) {
    double v[Z][PER];
#pragma unroll
    for (int z = 0; z < Z; ++z)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const double* q = p + min(z0 + z, a.slices - 1) * step + min(lane + 64 * i, a.n_experts - 1);
        if constexpr (DEVICE)
          v[z][i] = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else
          v[z][i] = *q;
      }
#pragma unroll
    for (int z = 0; z < Z; ++z)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (z0 + z < a.slices) l[i] += v[z][i];
  }
  if (a.logits_out != nullptr) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < a.n_experts) a.logits_out[(int64_t)t * a.n_experts + lane + 64 * i] = (float)l[i];
  }
  gate_select<PER>(a, t, l, bias, sc);
}

// Q8 blocks of columns lo .. hi - 1 of one row of x by the workgroup.
__device__ __forceinline__ void put_q8(const GateArgs& a, int t, int lo, int hi) {
  for (int c = lo + 4 * (int)threadIdx.x; c < hi; c += 4 * 64 * kGateWaves) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.x + t * a.ldx + c);
    const float vv[4] = {v[0], v[1], v[2], v[3]};
    float d;
    int sum;
    const uint32_t packed = q8_block8(vv, d, sum);
    *reinterpret_cast<uint32_t*>(a.qs + (int64_t)t * a.k + c) = packed;
    if ((threadIdx.x & 7) == 0) {
      a.qd[(int64_t)t * (a.k / 32) + c / 32] = d;
      a.qsum[(int64_t)t * (a.k / 32) + c / 32] = sum;
    }
  }
}

// Sums of N values over each 16 lanes: lane l has that of value l % N (while
// there are several, a lane keeps one half of them and gives the other away).
template <int H, int N>
__device__ __forceinline__ void fold16(double* v, int lane) {
  if constexpr (H >= 1) {
    constexpr int kCtrl = H == 8 ? DPP_MIRROR : (H == 4 ? DPP_HALF_MIRROR : (H == 2 ? DPP_XOR2 : DPP_XOR1));
    if constexpr (N > H) {
      static_assert(N == 2 * H, "N a power of two of at most 16");
      const bool hi = (lane & H) != 0;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const double send = hi ? v[j] : v[j + H];
        const double keep = hi ? v[j + H] : v[j];
        v[j] = keep + dpp_d<kCtrl>(send);
      }
      fold16<H / 2, N / 2>(v, lane);
    } else {
      static_assert(H >= N, "lanes above the values' hold the same ones");
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += dpp_d<kCtrl>(v[j]);
      fold16<H / 2, N>(v, lane);
    }
  }
}

}  // namespace

// Few tokens: a workgroup has kFewExperts experts and TG tokens, its waves the
// columns between them, four a lane; l in fp64, where products of fp32 numbers
// are exact.  The last workgroup to arrive chooses, a wave for each token.
template <int PER, int TG>
__global__ __launch_bounds__(64 * kGateWaves) void k_gate_few(GateArgs a) {
  constexpr int P = kFewExperts * TG;
  constexpr int kRed = kGateWaves * 4 * P, kSc = TG * 64 * PER;
  __shared__ double lds[kRed > kSc ? kRed : kSc];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = blockIdx.x * kFewExperts;
  double acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.0;
  for (int c = 4 * (int)threadIdx.x; c < a.k; c += 4 * 64 * kGateWaves) {
    f32x4 w[kFewExperts], x[TG];
#pragma unroll
    for (int e = 0; e < kFewExperts; ++e)
      w[e] = *reinterpret_cast<const f32x4*>(a.wr + (int64_t)min(e0 + e, a.n_experts - 1) * a.k + c);
#pragma unroll
    for (int t = 0; t < TG; ++t) x[t] = *reinterpret_cast<const f32x4*>(a.x + min(t, a.n_tok - 1) * a.ldx + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < kFewExperts; ++e)
#pragma unroll
        for (int t = 0; t < TG; ++t) acc[e * TG + t] = fma((double)w[e][i], (double)x[t][i], acc[e * TG + t]);
  }
  if (a.qs != nullptr && (int)blockIdx.x < a.n_tok) put_q8(a, blockIdx.x, 0, a.k);
  if (a.qs != nullptr && gridDim.x < a.n_tok && blockIdx.x == 0)  // fewer workgroups than tokens
    for (int t = gridDim.x; t < a.n_tok; ++t) put_q8(a, t, 0, a.k);
  fold16<8, P>(acc, lane);
  if ((lane & 15) < P) lds[(4 * wave + lane / 16) * P + (lane & 15)] = acc[0];
  __syncthreads();
  if (threadIdx.x < P) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4 * kGateWaves; ++i) s += lds[i * P + threadIdx.x];
    const int e = e0 + threadIdx.x / TG, t = threadIdx.x % TG;
    if (e < a.n_experts && t < a.n_tok)
      __hip_atomic_store(&a.logits[(int64_t)t * a.n_experts + e], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // Logits are device-scope atomic accesses (written through and reloaded by
  // the L2s), so waiting for this lane's own stores before the barrier and the
  // counter's update orders them without a device-scope fence.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.cnt, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  if (threadIdx.x == 0) atomicExch(a.cnt, 0);
  if (wave < a.n_tok) gate_token<PER, true>(a, wave, lds + wave * 64 * PER);  // no barrier in it
}

// More tokens: l on the fp64 matrix unit.  A workgroup has 16 experts and 16
// tokens, its waves deal the columns of its slice among themselves, 16 a step.
// A lane holds four neighbouring columns of one expert and of one token, of
// which each product takes one.
__global__ __launch_bounds__(64 * kGateWaves) void k_gate_logits(GateArgs a) {
  constexpr int kPad = kGateTile + 1;
  __shared__ double lds[kGateWaves * kGateTile * kPad];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * kGateTile, t0 = blockIdx.y * kGateTile;
  const int lo = blockIdx.z * a.slice, hi = min(lo + a.slice, a.k);
  const int at = 4 * (lane / 16);
  const float* w = a.wr + (int64_t)min(e0 + lane % 16, a.n_experts - 1) * a.k + at;
  const float* x = a.x + min(t0 + lane % 16, a.n_tok - 1) * a.ldx + at;
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  constexpr int kStep = 16 * kGateWaves;
  for (int c0 = lo + 16 * wave; c0 < hi; c0 += kGateAhead * kStep) {  // uniform
    f32x4 wv[kGateAhead], xv[kGateAhead];
#pragma unroll
    for (int u = 0; u < kGateAhead; ++u) {
      const int c = c0 + u * kStep;
      wv[u] = xv[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (c + at < hi) {
        wv[u] = *reinterpret_cast<const f32x4*>(w + c);
        xv[u] = *reinterpret_cast<const f32x4*>(x + c);
      }
    }
#pragma unroll
    for (int u = 0; u < kGateAhead; ++u)
      if (c0 + u * kStep < hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)wv[u][i], (double)xv[u][i], acc, 0, 0, 0);
      }
  }
  if (a.qs != nullptr)  // the slice's Q8 blocks, the tile's tokens dealt among the workgroups along the experts
    for (int t = t0 + blockIdx.x; t < min(t0 + kGateTile, a.n_tok); t += gridDim.x) put_q8(a, t, lo, hi);
  // element r of the product: expert 4 r + lane / 16, token lane % 16
#pragma unroll
  for (int r = 0; r < 4; ++r) lds[(wave * kGateTile + lane % 16) * kPad + 4 * r + lane / 16] = acc[r];
  __syncthreads();
  if (threadIdx.x < kGateTile * kGateTile) {
    const int e = threadIdx.x % kGateTile, t = threadIdx.x / kGateTile;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kGateWaves; ++i) s += lds[(i * kGateTile + t) * kPad + e];
    if (e0 + e < a.n_experts && t0 + t < a.n_tok)
      a.logits[((int64_t)blockIdx.z * a.n_tok + t0 + t) * a.n_experts + e0 + e] = s;
  }
}

// One wave a token.
template <int PER>
__global__ __launch_bounds__(64) void k_gate_select(GateArgs a) {
  __shared__ double sc[64 * PER];
  gate_token<PER, false>(a, blockIdx.x, sc);
}

int gate_slices(int64_t n_tok, int64_t n_experts) {
  // a workgroup for each compute unit
  const int64_t tiles = ((n_tok + kGateTile - 1) / kGateTile) * ((n_experts + kGateTile - 1) / kGateTile);
  const int64_t s = 256 / tiles;
  return (int)(s < 1 ? 1 : (s > kGateMaxSlices ? kGateMaxSlices : s));
}

// Several slices are of 256 tiles in all at most.
int64_t gate_room(int64_t n_tok, int64_t n_experts) {
  const int64_t one = n_tok * n_experts, most = one * kGateMaxSlices, sliced = 256 * kGateTile * kGateTile;
  return most < sliced ? most : (one > sliced ? one : sliced);
}

namespace {

template <int PER>
hipError_t launch(const GateArgs& a, hipStream_t st) {
  const dim3 block(64 * kGateWaves);
  if (a.n_tok <= 4) {
    const dim3 grid((unsigned)((a.n_experts + kFewExperts - 1) / kFewExperts));
    if (a.n_tok == 1) hipLaunchKernelGGL((k_gate_few<PER, 1>), grid, block, 0, st, a);
    else if (a.n_tok == 2) hipLaunchKernelGGL((k_gate_few<PER, 2>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_gate_few<PER, 4>), grid, block, 0, st, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.n_experts + kGateTile - 1) / kGateTile), (unsigned)((a.n_tok + kGateTile - 1) / kGateTile),
                  (unsigned)a.slices);
  hipLaunchKernelGGL(k_gate_logits, grid, block, 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_gate_select<PER>), dim3((unsigned)a.n_tok), dim3(64), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_gate(GateArgs a, hipStream_t st) {
  // slices in whole steps of all waves (which Q8 blocks are too), two for each wave or more
  constexpr int kStep = 16 * kGateWaves;
  const int steps = (a.k + kStep - 1) / kStep;
  a.slices = a.n_tok <= 4 ? 1 : min(gate_slices(a.n_tok, a.n_experts), (steps + 1) / 2);
  a.slice = (steps + a.slices - 1) / a.slices * kStep;
  a.slices = (a.k + a.slice - 1) / a.slice;
  const int per = (a.n_experts + 63) / 64;
  if (per <= 1) return launch<1>(a, st);
  if (per <= 2) return launch<2>(a, st);
  if (per <= 4) return launch<4>(a, st);
  if (per <= 8) return launch<8>(a, st);
  return launch<16>(a, st);
}

}  // namespace qmv
