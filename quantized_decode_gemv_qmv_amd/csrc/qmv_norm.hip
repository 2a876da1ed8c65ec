// qmv_norm.hip -- residual addition, root-mean-square norm and Q8 activation
// blocks in one pass, for gfx950.
#include "qmv_attn.h"
#include "qmv_device.h"

namespace qmv {

namespace {

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

// Sum over each 16-lane row; every lane of the row gets it.
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_d<DPP_XOR1>(v);
  v += dpp_d<DPP_XOR2>(v);
  v += dpp_d<DPP_HALF_MIRROR>(v);
  return v + dpp_d<DPP_MIRROR>(v);
}

}  // namespace

// r = x + res, y = (r * inv) * w with inv = 1 / sqrt(mean r^2 + eps), then the
// Q8 blocks of y as k_quantize makes them.  TPR threads hold one row in
// registers, NV 16-byte vectors each, so that x, res and w are read once and r
// and the blocks written once: 13.25 bytes a value, which bounds the kernel
// (8192 x 14336: 275 us, 5.66 TB/s; one row of 4096: 3.2 us, all latency).  Rows
// that stay in the caches are bound by the vector ALU: 1000 x 4128 takes 10.2 us,
// 7.1 of them vector instructions (some 200 a vector of four values: q8_block8
// divides and rounds each).
// Eight neighbouring lanes hold a block of 32 (q8_block8).  The squares are
// summed in fp64, where each is exact (the card's fp64 rate leaves the sum
// hidden behind the loads).  The sum's order could change it by some 2^-53 of
// itself a step, and so inv next to a border between two fp32 numbers; it
// depends on k alone, so a row gives the same bits wherever it stands.
// inv and both products are rounded to fp32.
template <int TPR, int NV, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(NormArgs a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;  // rows of a workgroup
  const int tid = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  if (RPW > 1 && row >= a.rows) return;  // no barrier below when a row is one wave
  const int nv = a.k / 4;
  const float* x = a.x + row * a.ldx;
  f32x4 r[NV], w[NV <= 4 ? NV : 1];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + TPR * j;
    r[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (i < nv) r[j] = *reinterpret_cast<const f32x4*>(x + 4 * i);
  }
  if constexpr (RES) {
    const float* res = a.res + row * a.ldr;
    f32x4 e[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + TPR * j;
      e[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i < nv) e[j] = *reinterpret_cast<const f32x4*>(res + 4 * i);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] += e[j];
  }
  // the weights' loads overlap the sum where registers allow
  constexpr bool EARLY = NV <= 4;
  if constexpr (EARLY) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + TPR * j;
      w[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i < nv) w[j] = *reinterpret_cast<const f32x4*>(a.w + 4 * i);
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) ss += (double)r[j][c] * (double)r[j][c];
  if (a.sum != nullptr) {
    float* so = a.sum + row * a.lds;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + TPR * j;
      if (i < nv) *reinterpret_cast<f32x4*>(so + 4 * i) = r[j];
    }
  }
  ss = row_sum(ss);
  ss = (lane_d(ss, 0) + lane_d(ss, 16)) + (lane_d(ss, 32) + lane_d(ss, 48));
  if constexpr (TPR > 64) {
    __shared__ double part[16];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    const int l = threadIdx.x & 15;
    ss = row_sum(l < TPR / 64 ? part[l] : 0.0);
  }
  const float inv = (float)(1.0 / sqrt(ss / (double)a.k + (double)a.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + TPR * j;
    if constexpr (!EARLY) __builtin_amdgcn_sched_barrier(0);  // one at a time: the registers hold the row
    if (i < nv) {  // all eight lanes of a block together: k is a multiple of 32
      float v[4];
      f32x4 wj;
      if constexpr (EARLY) wj = w[j];
      else wj = *reinterpret_cast<const f32x4*>(a.w + 4 * i);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = (r[j][c] * inv) * wj[c];
      float db;
      int sum;
      const uint32_t packed = q8_block8(v, db, sum);
      if (a.y != nullptr) *reinterpret_cast<f32x4*>(a.y + row * a.ldy + 4 * i) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<uint32_t*>(a.qs + row * a.k + 4 * i) = packed;
      if ((tid & 7) == 0) {
        const int64_t b = row * (a.k / 32) + i / 8;
        a.d[b] = db;
        a.s[b] = sum;
      }
    }
  }
}

namespace {

template <int TPR, int NV>
hipError_t launch(const NormArgs& a, hipStream_t st) {
  constexpr int T = TPR < 256 ? 256 : TPR, RPW = T / TPR;
  const unsigned grid = (unsigned)((a.rows + RPW - 1) / RPW);
  if (a.res != nullptr)
    hipLaunchKernelGGL((k_rmsnorm<TPR, NV, true>), dim3(grid), dim3(T), 0, st, a);
  else
    hipLaunchKernelGGL((k_rmsnorm<TPR, NV, false>), dim3(grid), dim3(T), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// Threads of a row by its length: one wave up to two 16-byte vectors each, 256
// and 512 threads up to two each, beyond that 1024.  Us at 1 / 64 / 2048 rows with a
// residual (256, 512, 1024 threads): 1024 values 2.1 / 2.4 / 7.8, 2.1 / 2.4 /
// 7.6, 2.2 / 2.4 / 9.0; 4096 values 4.0 / 4.4 / 25.9, 3.2 / 3.5 / 22.4, 3.3 /
// 3.7 / 23.5; 8192 values 11.8 / 12.7 / 89.7, 5.0 / 5.5 / 44.4, 4.6 / 5.1 /
// 43.8.  One wave a row saves the barrier where two vectors a lane hold it.
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  const int nv = a.k / 4;
  if (nv <= 64) return launch<64, 1>(a, st);
  if (nv <= 128) return launch<64, 2>(a, st);
  if (nv <= 256) return launch<256, 1>(a, st);
  if (nv <= 512) return launch<256, 2>(a, st);
  if (nv <= 1024) return launch<512, 2>(a, st);
  switch ((nv + 1023) / 1024) {
    case 2: return launch<1024, 2>(a, st);
    case 3: return launch<1024, 3>(a, st);
    case 4: return launch<1024, 4>(a, st);
    case 5:
    case 6:
    case 7:
    case 8: return launch<1024, 8>(a, st);
    case 9:
    case 10:
    case 11:
    case 12: return launch<1024, 12>(a, st);
    case 13:
    case 14:
    case 15:
    case 16: return launch<1024, 16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
