// qmv_logprobs.hip -- log probabilities of given tokens, entropy and the
// likeliest alternatives of the output head's logits in one pass, for gfx950.
//
// A row's softmax needs its largest value m, s = sum e^d and u = sum e^d d with
// d = scale x - scale m: log p = d - ln s, the entropy is ln s - u / s, whose
// terms all have one sign.  Partial sums over parts of a row join by their
// maxima.  The n largest come from the same pass: each group of elements gives
// its largest, the n-th largest of 64 groups of groups is a bound that n
// elements reach, and only groups whose largest reaches it are read again
// (some tens, from the caches).
//
// Many rows are bound by their bytes (1000 x 50257 with five alternatives 42.5 us,
// 4.7 TB/s), few by a chain: launch, load, sums, handoff to the row's last
// workgroup, keys, bound, second reading (6 x 152064 with twenty 8.2 us, without
// alternatives 5.7; 64 x 152064 20.9, with five 16.0, without 12.6).  512 threads a
// row let three rows share a compute unit, where 1024 let one (62.9 -> 41.7 us).
#include "qmv_device.h"
#include "qmv_steps.h"

// Sums are relative to m as it was rounded.  Fused into a product m = scale x, a
// difference from m would be one from the exact product, off by |m| 2^-24 each time.
#pragma clang fp contract(off)

namespace qmv {

namespace {

constexpr float kLog2e = 1.44269504f;
constexpr int kRowThreads = 512;   // of a workgroup that has a whole row
constexpr int kPartThreads = 512;  // of one that has a part, and may join the row
constexpr int kPartVecs = 2;       // 16-byte vectors of a thread
constexpr int kPartVec = kPartThreads * kPartVecs;  // vectors of a part
constexpr int kPartGroups = kPartThreads / 16;      // groups of 16 lanes
static_assert(kPartGroups == kPartGroupsOfRow, "the workspace holds a part's keys");
constexpr int64_t kPartTarget = 512;  // workgroups of a launch in parts, about
constexpr int kList = 1024;        // candidates, and groups, that LDS lists

// Order of logits as unsigned numbers: the larger value first, then the lower
// index; NaN counts as -inf, -0 as +0.  0 is below every key.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  if (!(v == v)) v = -__builtin_inff();
  uint32_t b = __float_as_uint(v + 0.f);
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
  return ((uint64_t)(uint32_t)dpp_i<CTRL>((int)(uint32_t)(v >> 32)) << 32) | (uint32_t)dpp_i<CTRL>((int)(uint32_t)v);
}
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The largest of each 16 lanes, in all of them.
__device__ __forceinline__ uint64_t row_max(uint64_t v) {
  v = max_u64(v, dpp_u64<DPP_XOR1>(v));
  v = max_u64(v, dpp_u64<DPP_XOR2>(v));
  v = max_u64(v, dpp_u64<DPP_HALF_MIRROR>(v));
  return max_u64(v, dpp_u64<DPP_MIRROR>(v));
}
__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = row_max(v);
  return max_u64(max_u64(lane_u64(v, 0), lane_u64(v, 16)), max_u64(lane_u64(v, 32), lane_u64(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max8(v);
  v = fmaxf(v, dpp_f<DPP_MIRROR>(v));
  const int b = __float_as_int(v);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}

// m: largest logit times scale; s and u: sums relative to it.
struct Sums {
  float m, s, u;
};

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// The sums taken relative to m (which is not below their own).  A part with
// nothing allowed has m -inf and sums of 0, which stay; NaN stays too.
__device__ __forceinline__ void shift(Sums& a, float m) {
  const float d = fmaxf(a.m - m, -1e4f);
  const float f = exp_of(d);
  a.u = f * fmaf(d, a.s, a.u);
  a.s *= f;
  a.m = m;
}

// Adds one vector's elements to sums relative to ref (finite).
__device__ __forceinline__ void add(float& s, float& u, const f32x4& v, float scale, float ref) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float d = fmaf(v[i], scale, -ref);
    const float e = exp_of(d);
    s += e;
    u = fmaf(e, fmaxf(d, -1e4f), u);  // 0 for -inf
  }
}

__device__ __forceinline__ float max4(const f32x4& v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }

// Vector i of a row: elements past its end are -inf.
__device__ __forceinline__ f32x4 load_vec(const float* row, int i, int n) {
  if (4 * i + 4 <= n) return *reinterpret_cast<const f32x4*>(row + 4 * i);
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 4 * i + j < n ? row[4 * i + j] : -__builtin_inff();
  return v;
}

// Joins the sums of a wave's lanes, then of a workgroup's waves, in all threads.
template <int THREADS>
__device__ __forceinline__ Sums block_join(Sums a, Sums* tmp) {
  const float m = wave_max(a.m);
  shift(a, m);
  a.s = wave_sum(a.s);
  a.u = wave_sum(a.u);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = a;
  __syncthreads();
  Sums r = tmp[0];
  float top = r.m;
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) top = fmaxf(top, tmp[w].m);
  shift(r, top);
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) {
    Sums o = tmp[w];
    shift(o, top);
    r.s += o.s;
    r.u += o.u;
  }
  return r;
}

__device__ __forceinline__ float log_prob(float x, float scale, const Sums& a, double log_s) {
  if (a.m == -__builtin_inff() && a.s == 0.f) return -__builtin_inff();  // nothing is allowed
  return (float)(((double)x * (double)scale - (double)a.m) - log_s);
}

// The given token that a thread starts with, and its logit.
struct Given {
  int id;
  float x;
};
__device__ __forceinline__ Given first_given(const LogprobArgs& a, int t, const float* row) {
  Given g{-1, 0.f};
  if ((int)threadIdx.x < a.n_given) g.id = a.given[(int64_t)t * a.n_given + threadIdx.x];
  if (g.id >= 0 && g.id < a.n_vocab) g.x = row[g.id];
  return g;
}

// Entropy and the given tokens' log probabilities of row t.
template <int THREADS>
__device__ __forceinline__ void put_given(const LogprobArgs& a, int t, const float* row, const Sums& r, double log_s,
                                          Given g) {
  if (threadIdx.x == 0 && a.entropy != nullptr) {
    const bool none = r.m == -__builtin_inff() && r.s == 0.f;
    a.entropy[t] = none ? 0.f : (float)(log_s - (double)r.u / (double)r.s);
  }
  // sums are NaN where the row holds NaN or +inf, and m is inf where a z is
  const float outside = r.s == r.s && r.m < __builtin_inff() ? -__builtin_inff() : __builtin_nanf("");
  for (int i = threadIdx.x; i < a.n_given; i += THREADS) {
    const int64_t at = (int64_t)t * a.n_given + i;
    if (i != (int)threadIdx.x) {
      g.id = a.given[at];
      if (g.id >= 0 && g.id < a.n_vocab) g.x = row[g.id];
    }
    a.logprobs[at] = g.id < 0 || g.id >= a.n_vocab ? outside : log_prob(g.x, a.scale, r, log_s);
  }
}

struct TopShared {
  uint64_t coarse[64];
  uint64_t key[kList];
  uint64_t wave[8];
  uint64_t least;
  uint32_t group[kList];
  int groups, keys;
};

// The n-th largest of the largest keys of 64 groups of neighbouring threads
// (0 where fewer are above 0; the others are all different), in every thread.
template <int THREADS>
__device__ __forceinline__ uint64_t bound(uint64_t k, int n, TopShared& sh) {
  constexpr int L = THREADS / 64;  // threads of a group
  static_assert(L == 8, "a group is eight lanes, a workgroup eight waves");
  const int tid = threadIdx.x;
  k = max_u64(k, dpp_u64<DPP_XOR1>(k));
  k = max_u64(k, dpp_u64<DPP_XOR2>(k));
  k = max_u64(k, dpp_u64<DPP_HALF_MIRROR>(k));
  if (tid % L == 0) sh.coarse[tid / L] = k;
  if (tid == 0) {
    sh.least = 0;
    sh.groups = sh.keys = 0;
  }
  __syncthreads();
  // a group's threads compare its key with 64 / L others each
  int larger = 0;
#pragma unroll
  for (int j = 0; j < 64 / L; ++j) larger += sh.coarse[j * L + tid % L] > k ? 1 : 0;
  larger = sum8(larger);
  if (tid % L == 0 && larger == n - 1 && k != 0) sh.least = k;
  __syncthreads();
  return sh.least;
}

// The n largest of a row by the threads that hold its groups' largest keys
// (mine: the largest of this thread's groups).  each(f) calls f(key, group) for
// the thread's groups; vec(list, q), q < count(groups), is the q-th vector of the
// listed groups.  A group's key is its largest value's, with the last index of
// the vector where that value first stands.
template <int THREADS, class Each, class Count, class Vec>
__device__ void put_top(const LogprobArgs& a, int t, const float* row, const Sums& r, double log_s, uint64_t mine,
                        TopShared& sh, Each each, Count count_of, Vec vec) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.top_n;
  uint64_t least = bound<THREADS>(mine, n, sh);
  each([&](uint64_t k, uint32_t g) {
    if (k != 0 && k >= least) {
      const int at = atomicAdd(&sh.groups, 1);
      if (at < kList) sh.group[at] = g;
    }
  });
  __syncthreads();
  const int n_groups = sh.groups;
  const bool listed = n_groups <= kList;
  // all vectors that may hold one: of the listed groups, or of the row
  const int count = listed ? count_of(n_groups) : (a.n_vocab + 3) / 4;
  auto scan = [&](auto f) {
    for (int q = tid; q < count; q += THREADS) {
      const int i = listed ? vec(sh.group, q, n_groups) : q;
      if (4 * i >= a.n_vocab) continue;
      const f32x4 v = load_vec(row, i, a.n_vocab);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * i + j < a.n_vocab) f(key_of(v[j], (uint32_t)(4 * i + j)));
    }
  };
  uint64_t top = 0;
  scan([&](uint64_t k) {
    if (k >= least) {
      top = max_u64(top, k);
      const int at = atomicAdd(&sh.keys, 1);
      if (at < kList) sh.key[at] = k;
    }
  });
  __syncthreads();
  if (sh.keys > kList) {  // once more with the bound that these themselves give
    __syncthreads();
    least = max_u64(least, bound<THREADS>(top, n, sh));
    scan([&](uint64_t k) {
      if (k >= least) {
        const int at = atomicAdd(&sh.keys, 1);
        if (at < kList) sh.key[at] = k;
      }
    });
    __syncthreads();
  }
  const int c = sh.keys;
  auto put = [&](int j, uint64_t k) {
    a.ids[(int64_t)t * n + j] = (int)~(uint32_t)k;
    a.top[(int64_t)t * n + j] = log_prob(value_of(k), a.scale, r, log_s);
  };
  if (c <= THREADS / 2) {  // each one's place is the number of larger ones; eight threads count
    for (int i = tid / 8; i < (c + THREADS / 8 - 1) / (THREADS / 8) * (THREADS / 8); i += THREADS / 8) {  // uniform trips
      const uint64_t k = i < c ? sh.key[i] : 0;
      int larger = 0;
      for (int j = tid & 7; j < c; j += 8) larger += sh.key[j] > k ? 1 : 0;
      larger = sum8(larger);
      if ((tid & 7) == 0 && k != 0 && larger < n) put(larger, k);
    }
  } else if (c <= kList) {  // one after the other, by one wave
    if (wave == 0) {
      uint64_t k[kList / 64];
#pragma unroll
      for (int i = 0; i < kList / 64; ++i) k[i] = lane + 64 * i < c ? sh.key[lane + 64 * i] : 0;
      uint64_t last = ~0ull;
      for (int j = 0; j < n; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kList / 64; ++i) best = k[i] < last ? max_u64(best, k[i]) : best;
        last = wave_max(best);
        if (lane == 0) put(j, last);
      }
    }
  } else {  // too many that the bounds cannot tell apart: a scan for each
    uint64_t last = ~0ull;
    for (int j = 0; j < n; ++j) {
      uint64_t best = 0;
      scan([&](uint64_t k) { best = k < last ? max_u64(best, k) : best; });
      best = wave_max(best);
      __syncthreads();
      if (lane == 0) sh.wave[wave] = best;
      __syncthreads();
      last = row_max(sh.wave[lane & (THREADS / 64 - 1)]);
      if (tid == 0) put(j, last);
    }
  }
}

// A thread's vectors i0, i0 + THREADS .. below end, four a step: its largest logit
// and the vector where that first stands, and its sums relative to its own largest.
template <int THREADS>
__device__ __forceinline__ void take(const float* row, int i0, int end, int n, float scale, float& top, int& at, Sums& r) {
  constexpr int B = 4;
  for (int i1 = i0; i1 < end; i1 += B * THREADS) {
    f32x4 v[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = i1 + b * THREADS;
      v[b] = f32x4{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
      if (i < end) v[b] = load_vec(row, i, n);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float m = max4(v[b]);
      if (m > top) {
        top = m;
        at = i1 + b * THREADS;
      }
    }
    const float m = top * scale;
    shift(r, m);
    const float ref = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
    for (int b = 0; b < B; ++b) add(r.s, r.u, v[b], scale, ref);
  }
}

}  // namespace

// A whole row by one workgroup: each thread keeps sums relative to its own
// largest, four vectors a step.
__global__ __launch_bounds__(kRowThreads) void k_logprob_row(LogprobArgs a) {
  __shared__ Sums tmp[kRowThreads / 64];
  __shared__ TopShared sh;
  const int t = blockIdx.x, tid = threadIdx.x;
  const float* row = a.x + t * a.ldx;
  const int vecs = (a.n_vocab + 3) / 4;
  const Given given = first_given(a, t, row);
  float top = -__builtin_inff();
  int at = tid;
  Sums r{-__builtin_inff(), 0.f, 0.f};
  take<kRowThreads>(row, tid, vecs, a.n_vocab, a.scale, top, at, r);
  r = block_join<kRowThreads>(r, tmp);
  const double log_s = log((double)r.s);
  put_given<kRowThreads>(a, t, row, r, log_s, given);
  if (a.top_n > 0) {
    const uint64_t key = tid < vecs ? key_of(top, (uint32_t)(4 * at + 3)) : 0;
    const int items = (vecs + kRowThreads - 1) / kRowThreads;
    put_top<kRowThreads>(a, t, row, r, log_s, key, sh, [&](auto f) { f(key, (uint32_t)tid); },
                         [&](int groups) { return groups * items; },
                         [](const uint32_t* list, int q, int groups) {
                           return (int)(list[(uint32_t)q % (uint32_t)groups] + (uint32_t)q / (uint32_t)groups * kRowThreads);
                         });
  }
}

namespace {

__device__ __forceinline__ void put_device(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_device(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

// One part of a row: its sums and the largest of each 16 lanes' vectors.  The last
// workgroup of a row to arrive joins its parts.  A part is held in registers, or,
// with MANY, a.loops times as long.
template <bool MANY>
__global__ __launch_bounds__(kPartThreads) void k_logprob_part(LogprobArgs a) {
  __shared__ Sums tmp[kPartThreads / 64];
  __shared__ TopShared sh;
  __shared__ int s_last;
  const int t = blockIdx.y, p = blockIdx.x, tid = threadIdx.x;
  const float* row = a.x + t * a.ldx;
  const int loops = MANY ? a.loops : 1, span = loops * kPartVec;
  const int vecs = (a.n_vocab + 3) / 4, i0 = p * span + tid;
  float top = -__builtin_inff();
  int at = i0;
  Sums r{-__builtin_inff(), 0.f, 0.f};
  if constexpr (MANY) {
    take<kPartThreads>(row, i0, min((p + 1) * span, vecs), a.n_vocab, a.scale, top, at, r);
  } else {
    f32x4 v[kPartVecs];
#pragma unroll
    for (int b = 0; b < kPartVecs; ++b) {
      const int i = i0 + b * kPartThreads;
      v[b] = f32x4{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
      if (i < vecs) v[b] = load_vec(row, i, a.n_vocab);
    }
#pragma unroll
    for (int b = 0; b < kPartVecs; ++b) {
      const float m = max4(v[b]);
      if (m > top) {
        top = m;
        at = i0 + b * kPartThreads;
      }
    }
    const float m = wave_max(top) * a.scale;
    const float ref = m == -__builtin_inff() ? 0.f : m;
    r.m = m;
#pragma unroll
    for (int b = 0; b < kPartVecs; ++b) add(r.s, r.u, v[b], a.scale, ref);
  }
  uint64_t* keys = a.keys + (int64_t)t * a.parts * kPartGroups;
  uint64_t* sums = reinterpret_cast<uint64_t*>(a.sums) + 2 * (int64_t)t * a.parts;
  if (a.top_n > 0) {
    const uint64_t key = row_max(i0 < vecs ? key_of(top, (uint32_t)(4 * at + 3)) : 0);
    if ((tid & 15) == 0) put_device(keys + p * kPartGroups + (tid >> 4), key);
  }
  r = block_join<kPartThreads>(r, tmp);
  if (tid == 0) {
    put_device(sums + 2 * p, ((uint64_t)__float_as_uint(r.s) << 32) | __float_as_uint(r.m));
    put_device(sums + 2 * p + 1, __float_as_uint(r.u));
  }
  // Keys and sums are device-scope atomic accesses (written through and
  // reloaded by the L2s), so waiting for this lane's own stores before the
  // barrier and the counter's update orders them without a device-scope fence.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.cnt[t * kCounterStep], 1) == a.parts - 1;
  __syncthreads();
  if (!s_last) return;
  if (tid == 0) atomicExch(&a.cnt[t * kCounterStep], 0);
  // what each later step needs first, on its way together.  The bound's groups are
  // neighbouring threads: those of few keys hold some 64 apart, so that each group
  // has its share (neighbouring keys fill 4 groups a part, and a bound of more
  // alternatives than groups is none: 128 rows of 262144, 4 parts, twenty
  // alternatives 271 us against 45)
  const Given given = first_given(a, t, row);
  const int groups = a.parts * kPartGroups;
  const int k0 = groups < kPartThreads ? tid % 8 * 64 + tid / 8 : tid;
  uint64_t first[3] = {0, 0, 0};
  if (a.top_n > 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (k0 + i * kPartThreads < groups) first[i] = get_device(keys + k0 + i * kPartThreads);
  }
  r = Sums{-__builtin_inff(), 0.f, 0.f};
  for (int i = tid; i < a.parts; i += kPartThreads) {
    const uint64_t ms = get_device(sums + 2 * i), u = get_device(sums + 2 * i + 1);
    Sums q{__uint_as_float((uint32_t)ms), __uint_as_float((uint32_t)(ms >> 32)), __uint_as_float((uint32_t)u)};
    const float big = fmaxf(q.m, r.m);
    shift(q, big);
    shift(r, big);
    r.s += q.s;
    r.u += q.u;
  }
  r = block_join<kPartThreads>(r, tmp);
  const double log_s = log((double)r.s);
  put_given<kPartThreads>(a, t, row, r, log_s, given);
  if (a.top_n == 0) return;
  uint64_t mine = max_u64(max_u64(first[0], first[1]), first[2]);
  for (int g = k0 + 3 * kPartThreads; g < groups; g += kPartThreads) mine = max_u64(mine, get_device(keys + g));
  put_top<kPartThreads>(a, t, row, r, log_s, mine, sh,
                        [&](auto f) {
#pragma unroll
                          for (int i = 0; i < 3; ++i) f(first[i], (uint32_t)(k0 + i * kPartThreads));
                          for (int g = k0 + 3 * kPartThreads; g < groups; g += kPartThreads)
                            f(get_device(keys + g), (uint32_t)g);
                        },
                        [=](int listed) { return listed * loops * kPartVecs * 16; },
                        [=](const uint32_t* list, int q, int) {
                          const uint32_t each = loops * kPartVecs * 16;  // vectors of a group
                          const int g = (int)list[(uint32_t)q / each], i = (int)((uint32_t)q % each);
                          return g / kPartGroups * span + (i >> 4) * kPartThreads + g % kPartGroups * 16 + (i & 15);
                        });
}

// Rows are shared by workgroups where that is not slower than whole rows, which
// leave compute units idle: rows of more than 2^15 tokens, and fewer rows the more
// alternatives there are, since a row's last workgroup reads n groups again that
// are as long as its parts.  Us as whole rows / in parts, without alternatives, with
// 5, 20 and 32: 41 rows of 50257 tokens 8.6 / 6.6, 10.3 / 9.0, 11.1 / 11.1, 11.9 /
// 14.1; 66 of 128256 17.6 / 11.5, 19.4 / 14.8, 21.0 / 19.4, 23.0 / 24.5; 126 of 152064
// 20.7 / 20.4, 22.7 / 25.5, 25.5 / 35.0, 28.1 / 43.5; 128 of 262144 32.7 / 25.6, 35.0 /
// 31.5, 39.9 / 45.2, 44.6 / 58.2.  Where the rule below takes parts they took 5 % longer
// than whole rows at most (33000 to 10^6 tokens, 0 to 32 alternatives).
// Parts are as long as some 512 workgroups leave them (256 / 512 / 768: 64 rows of
// 152064 16.4 / 15.8 / 16.8), and a row has four at least, whose 128 keys the
// alternatives' bound needs.
static int64_t part_loops(int64_t n_tok, int64_t n_vocab) {
  const int64_t most = (n_vocab + 4 * kPartVec - 1) / (4 * kPartVec);  // parts
  const int64_t loops = (n_tok * most + kPartTarget - 1) / kPartTarget;
  return loops < most / 4 ? loops : most / 4;
}
int logprob_parts(int64_t n_tok, int64_t n_vocab, int64_t top_n) {
  if (n_vocab <= 32768 || n_tok > kLogprobCounters ||  // a row in parts has a counter
      n_tok * (1200 + 20 * top_n) > n_vocab ||
      n_tok * (top_n > 0 ? 30 + top_n : 25) > 3300 + n_vocab / 400)
    return 0;
  const int64_t part = 4 * kPartVec * part_loops(n_tok, n_vocab);
  return (int)((n_vocab + part - 1) / part);
}

// A row has `most` parts, or as many as make kPartTarget in all and one a row, or,
// where loops are most / 4, six at most (most is 9 or more).
int64_t logprob_room(int64_t n_tok, int64_t n_vocab) {
  if (n_vocab <= 32768) return 0;
  const int64_t rows = n_tok * 1200 <= n_vocab ? n_tok : n_vocab / 1200;
  const int64_t most = rows * ((n_vocab + 4 * kPartVec - 1) / (4 * kPartVec));
  const int64_t target = rows + kPartTarget, few = 6 * rows;
  const int64_t longer = target > few ? target : few;
  return most < longer ? most : longer;
}

hipError_t launch_token_logprobs(LogprobArgs a, hipStream_t st) {
  if (a.parts == 0) {
    hipLaunchKernelGGL(k_logprob_row, dim3((unsigned)a.n_tok), dim3(kRowThreads), 0, st, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)a.parts, (unsigned)a.n_tok);
  a.loops = (int)part_loops(a.n_tok, a.n_vocab);
  if (a.loops > 1)
    hipLaunchKernelGGL(k_logprob_part<true>, grid, dim3(kPartThreads), 0, st, a);
  else
    hipLaunchKernelGGL(k_logprob_part<false>, grid, dim3(kPartThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace qmv
