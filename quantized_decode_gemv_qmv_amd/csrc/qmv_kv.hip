// qmv_kv.hip -- writing new keys and values into the 8-bit block cache, for
// gfx950.
#include "qmv_attn.h"
#include "qmv_device.h"

namespace qmv {

namespace {

// Whole number nearest to x, halves away from zero, within +-127.
__device__ __forceinline__ int code_of(float x) {
  // plus the number below a half, towards zero: below 2^22 a sum that should
  // not reach the next whole number does not round to it
  const int r = static_cast<int>(x + copysignf(0.49999997f, x));
  return r > 127 ? 127 : (r < -127 ? -127 : r);
}

// y / d, correctly rounded where it decides a code: from the reciprocal and, by
// Markstein's theorem, one step with the exact remainder (a third of a
// division's instructions, which had bounded the append of many tokens).  The
// theorem wants a quotient within one step of the true one, which y * inv is
// not for every y and d; so the five values of y about the middle between two
// codes were compared with a division for every fraction of d and every code:
// all 5.3e9 are equal.  d within 2^-100 .. 2^100.
struct Quotient {
  float d, inv;
  bool near;
  __device__ __forceinline__ explicit Quotient(float x) : d(x), inv(1.f / x), near(x > 1e-30f && x < 1e30f) {}
  __device__ __forceinline__ float operator()(float y) const {
    const float q = y * inv;
    return fmaf(fmaf(-q, d, y), inv, q);
  }
};

__device__ __forceinline__ float wave_max(float v) {
  v = max8(v);
  v = fmaxf(v, dpp_f<DPP_MIRROR>(v));
  const int b = __float_as_int(v);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}

__device__ __forceinline__ uint32_t pack4(const int (&c)[4]) {
  return (uint32_t)(c[0] & 255) | ((uint32_t)(c[1] & 255) << 8) | ((uint32_t)(c[2] & 255) << 16) |
         ((uint32_t)(c[3] & 255) << 24);
}

// New tokens of a sequence up to which both parts are written a token at a time.
constexpr int kFew = 16;

}  // namespace

// One workgroup per (sequence, head, K or V, cache block that gets new
// tokens).  The block's scale is d = max(d_old, amax / 127) over the new
// values, d_old counting only when tokens stand before the new ones; if it
// grew, the codes before them become round(q * (d_old / d)).  A thread keeps
// its new values in registers between the maximum and the codes, so they are
// read once.  K is stored [slot][dim]: neighbouring lanes take neighbouring
// quads of one token.  V is stored [dim][slot] (the attention kernel's second
// product reads 16 keys of one dim from one lane): a thread takes a square of
// four dims by four slots, 16 lanes along the slots, so that loads and stores
// both move 64 contiguous bytes.  Bytes of slots behind the new tokens are not
// written.  dim <= 64 * NI.  FEW: at most kFew new tokens a sequence, V taken as
// K is, its codes stored byte by byte: a thread then holds a sixteenth of a
// block's values at most, and does no work for slots without a new token (us
// with / without: 16 sequences, 8 heads, 128 dims, one new token 3.2 / 5.6, 256
// dims 4.1 / 8.9; 8 sequences of 16 3.9 / 6.4).
// Bound: with few tokens by the launch and two loads in a row (id and length,
// then the values; 16 x 1: 2.8 us); many by bytes (4 sequences of 2000, 8 heads,
// 128 dims: 16.7 us, 4.9 TB/s of values and codes, the rate of a large copy; with
// a division a value 19.7).  A block whose scale grows adds 2 us, its older codes'
// way there and back (16 x 1 behind 40 tokens 2.1 -> 4.1).
template <int NI, bool FEW>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
  const KvView& kv = a.kv;
  const int seq = blockIdx.z, head = blockIdx.y >> 1, part = blockIdx.y & 1;
  int t0 = seq * kv.max_q, n = kv.max_q;
  if (kv.start != nullptr) {
    t0 = min(max(kv.start[seq], 0), kv.n_tok);
    n = min(max(kv.start[seq + 1], t0), kv.n_tok) - t0;
    n = min(n, kv.max_q);
  }
  const int len = max(kv.lens[seq], 0);
  const int first = max(len - n, 0);  // position of the first new token kept
  const int b = first / 64 + (int)blockIdx.x;
  if (n < 1 || b >= kv.width) return;
  const int lo = max(first, 64 * b), hi = min(len, 64 * b + 64);
  if (lo >= hi) return;
  const int id = kv.table[(int64_t)seq * kv.width + b];
  const int s0 = lo - 64 * b, s1 = hi - 64 * b;  // slots [s0, s1) are new
  const int dim = kv.dim, qd = dim / 4;
  // x of slot j: token t0 + (64 b + j) - (len - n)
  const float* x = (part ? a.x[1] : a.x[0]) + head * (int64_t)dim;
  const int64_t ld = part ? a.ld[1] : a.ld[0];
  const int64_t tok0 = (int64_t)t0 + 64 * b - (len - n);

  constexpr int NV = FEW ? NI : 4 * NI;  // quads of a token that a thread holds
  f32x4 v[NV];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    int slot, quad;
    if (FEW || part == 0) {
      const int f = threadIdx.x + 256 * i;
      slot = s0 + f / qd;
      quad = f % qd;
    } else {
      slot = 4 * (threadIdx.x & 15) + (i & 3);
      quad = (threadIdx.x >> 4) + 16 * (i >> 2);
    }
    v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (slot >= s0 && slot < s1 && quad < qd) v[i] = *reinterpret_cast<const f32x4*>(x + (tok0 + slot) * ld + 4 * quad);
  }
  // the id's load was issued before the values'
  if (id < 0 || id >= kv.n_blocks) return;
  const int64_t plane = ((int64_t)id * 2 + part) * kv.kvh + head;
  const float old = s0 > 0 ? kv.scales[plane] : 0.f;
  __shared__ float part_max[4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) amax = fmaxf(amax, fabsf(v[i][c]));
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) part_max[threadIdx.x >> 6] = amax;
  __syncthreads();  // also: every thread has read the old scale before one writes the new one
  amax = fmaxf(fmaxf(part_max[0], part_max[1]), fmaxf(part_max[2], part_max[3]));
  const float d = fmaxf(old, amax / 127.0f);
  int8_t* codes = kv.codes + plane * (64 * (int64_t)dim);
  if (threadIdx.x == 0) kv.scales[plane] = d;

  const Quotient over(d);
  if (over.near) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) v[i][c] = over(v[i][c]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) v[i][c] = d > 0.f ? v[i][c] / d : 0.f;
  }
  if (FEW || part == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int f = threadIdx.x + 256 * i;
      const int slot = s0 + f / qd, quad = f % qd;
      const int c[4] = {code_of(v[i][0]), code_of(v[i][1]), code_of(v[i][2]), code_of(v[i][3])};
      if (slot >= s1) continue;
      if (part == 0) {
        *reinterpret_cast<uint32_t*>(codes + slot * dim + 4 * quad) = pack4(c);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) codes[(4 * quad + e) * 64 + slot] = (int8_t)c[e];
      }
    }
  } else if constexpr (!FEW) {
    const int slot = 4 * (threadIdx.x & 15);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int quad = (threadIdx.x >> 4) + 16 * i;
      if (quad >= qd || slot + 3 < s0 || slot >= s1) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        int8_t* at = codes + (4 * quad + c) * 64 + slot;
        const int q[4] = {code_of(v[4 * i][c]), code_of(v[4 * i + 1][c]), code_of(v[4 * i + 2][c]),
                          code_of(v[4 * i + 3][c])};
        if (slot >= s0 && slot + 4 <= s1) {
          *reinterpret_cast<uint32_t*>(at) = pack4(q);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (slot + e >= s0 && slot + e < s1) at[e] = (int8_t)q[e];
        }
      }
    }
  }
  if (s0 == 0 || !(old >= 0.f && d > old)) return;
  // the scale grew: the codes of slots [0, s0) in units of the new one; from a
  // scale of zero they become zeros, whatever they were
  const float ratio = old / d;
  if (part == 0) {
    for (int f = threadIdx.x; f < s0 * qd; f += 256) {
      uint32_t* at = reinterpret_cast<uint32_t*>(codes) + f;
      const uint32_t w = *at;
      int c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = code_of((float)(int8_t)(w >> (8 * e)) * ratio);
      *at = pack4(c);
    }
  } else {
    const int slot = 4 * (threadIdx.x & 15);
    if (slot >= s0) return;
    for (int r = threadIdx.x >> 4; r < dim; r += 16) {
      int8_t* at = codes + r * 64 + slot;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
      int c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = code_of((float)(int8_t)(w >> (8 * e)) * ratio);
      if (slot + 4 <= s0) {
        *reinterpret_cast<uint32_t*>(at) = pack4(c);
      } else {  // the dword in which the new tokens begin: their bytes are written above
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (slot + e < s0) at[e] = (int8_t)c[e];
      }
    }
  }
}

namespace {

template <int NI>
hipError_t launch(const AppendArgs& a, hipStream_t st) {
  // blocks that max_q tokens can touch, beginning anywhere in one
  const unsigned nb = (unsigned)((a.kv.max_q + 62) / 64 + 1);
  const dim3 grid(nb, (unsigned)(2 * a.kv.kvh), (unsigned)a.kv.n_seqs);
  if (a.kv.max_q <= kFew)
    hipLaunchKernelGGL((k_kv_append<NI, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_kv_append<NI, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t st) {
  if (a.kv.dim <= 64) return launch<1>(a, st);
  if (a.kv.dim <= 128) return launch<2>(a, st);
  return launch<4>(a, st);
}

}  // namespace qmv
