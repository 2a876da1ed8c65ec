// qmv_attn.hip -- attention of new tokens over the 8-bit block cache, for
// gfx950.
#include "qmv_attn.h"
#include "qmv_device.h"

namespace qmv {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Largest whole number a 24-bit operand holds: 127 * 2^16, so that its three
// base-256 digits all lie within -128..127.
constexpr float kTop = 8323072.0f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ i32x4 mfma(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48; all get it.
__device__ __forceinline__ float max4(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add4(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The base-256 digits of four whole numbers x (as x + 0x808080 in the low 24
// bits of u): dword e of d[] gets digit e of all four.  x + 0x808080 has the
// digits of x, each plus 128, as its bytes; the XOR takes the 128 off again.
__device__ __forceinline__ void digits4(const uint32_t (&u)[4], int& lo, int& mid, int& hi) {
  const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400);  // u0.b0 u1.b0 u0.b1 u1.b1
  const uint32_t b = __builtin_amdgcn_perm(u[3], u[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0602);  // u0.b2 u1.b2
  const uint32_t e = __builtin_amdgcn_perm(u[3], u[2], 0x06020c0c);
  lo = (int)(__builtin_amdgcn_perm(b, a, 0x05040100) ^ 0x80808080u);
  mid = (int)(__builtin_amdgcn_perm(b, a, 0x07060302) ^ 0x80808080u);
  hi = (int)((c | e) ^ 0x80808080u);
}

struct Group {
  int seq, head, rb;  // sequence, kv head, row block
  int t0, n, len;     // first token, new tokens, length
};

__device__ __forceinline__ Group group_of(const AttnArgs& a, int id) {
  Group g;
  g.rb = id % a.row_blocks;
  const int z = id / a.row_blocks;
  g.head = z % a.kv.kvh;
  g.seq = z / a.kv.kvh;
  g.t0 = g.seq * a.kv.max_q;
  g.n = a.kv.max_q;
  if (a.kv.start != nullptr) {
    g.t0 = min(max(a.kv.start[g.seq], 0), a.kv.n_tok);
    g.n = min(max(a.kv.start[g.seq + 1], g.t0), a.kv.n_tok) - g.t0;
    g.n = min(g.n, a.kv.max_q);
  }
  g.len = max(a.kv.lens[g.seq], 0);
  return g;
}

// Stores four values of one output row, and their Q8 block with the eight
// lanes that hold it.
__device__ __forceinline__ void store4(const AttnArgs& a, const Group& g, int row, int d, const float (&v)[4]) {
  const int64_t tok = g.t0 + row / a.group;
  const int col = (g.head * a.group + row % a.group) * a.kv.dim + d;
  if (a.out != nullptr) *reinterpret_cast<f32x4*>(a.out + tok * a.ldo + col) = f32x4{v[0], v[1], v[2], v[3]};
  if (a.qs != nullptr) {
    const int64_t width = (int64_t)a.kv.kvh * a.group * a.kv.dim;
    float db;
    int sum;
    const uint32_t packed = q8_block8(v, db, sum);
    *reinterpret_cast<uint32_t*>(a.qs + tok * width + col) = packed;
    if ((threadIdx.x & 7) == 0) {
      a.qd[tok * (width / 32) + col / 32] = db;
      a.qsum[tok * (width / 32) + col / 32] = sum;
    }
  }
}

}  // namespace

// Attention of the rows (new token, query head) of one (sequence, kv head)
// over its cache blocks, on int8 matrix instructions that read the cached
// codes as they are.
//
//   S = scale dq dk (Q K), P = exp(S - m), O = sum dv (P V)
//
// K and V hold int8 codes with one scale a block of 64 tokens.  The other
// operand of each product is taken in 24 bits: a row of q in units of its
// largest value / kTop, the weights P of one cache block in units of the
// row's largest weight in that block / kTop, each as three base-256 digits,
// so that a product is three exact integer products; their sums meet in fp32.
// The result is as near as fp32 arithmetic's (2^-24 of the largest value),
// and no code is ever converted.  The scales of a block are one number for
// the whole 64-key product, which is what they are chosen for.
//
// v_mfma_i32_16x16x64_i8: lane l supplies 16 bytes of A row l % 16 and of B
// column l % 16 for k = 16 (l / 16) .., and gets D[4 (l / 16) + r][l % 16].
// Scores are computed as S^T = K q^T with key 16 (m / 4) + 4 t + m % 4 in row
// m of product t: lane l then holds the scores of row l % 16 and of keys
// 16 (l / 16) .. + 15 in order, which are just the 16 bytes it supplies as
// the B operand of O^T = V^T P^T.  So P never leaves its lane, maxima and
// totals are a lane's own (but for two lane swaps), and V^T, stored [dim][64]
// in the cache, is loaded 16 bytes a lane.  O^T gives a lane four dims of its
// row at a time.
//
// A wave owns MR tiles of 16 rows; a workgroup's four waves are a.wr along the
// rows and 4 / a.wr along the cache blocks, and a.splits workgroups share a
// group's blocks.  The waves' sums meet in LDS in wave order, the workgroups'
// through the workspace: the last one to arrive adds them in split order, so
// the result does not depend on timing.  KS: 64-value steps of the head
// dimension; FULL: the dimension is all of them.  Bound by the cache's bytes for a few rows, by the vector ALU
// (about 450 instructions a tile of 16 rows and 64 keys at 128 dims) for many.
template <int KS, int MR, bool FULL>
__global__ __launch_bounds__(256, KS * MR <= 4 ? 2 : 1) void k_kv_attn(AttnArgs a) {
  constexpr int DT = 4 * KS;          // 16-dim tiles of the output
  constexpr int LD = 64 * KS + 4;     // LDS row stride (floats)
  extern __shared__ float lds[];      // [4 waves][16 rows][LD], then [4][16][2]
  float* lds_ml = lds + 4 * 16 * LD;
  const KvView& kv = a.kv;
  const int dim = FULL ? 64 * KS : kv.dim;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c16 = lane & 15, g4 = lane >> 4;
  const int split = blockIdx.x % a.splits, gid = blockIdx.x / a.splits;
  const Group g = group_of(a, gid);
  const int rows = g.n * a.group;
  const int wr = a.wr, wk = 4 / wr;
  const int my_r = wave % wr, my_k = wave / wr;
  const int wg_rows = wr * MR * 16;
  const int r0 = g.rb * wg_rows;
  if (r0 >= rows) return;
  const int base = g.len - g.n;  // position of the sequence's first new token

  // cache blocks that some row of the workgroup sees, and this split's share
  const int top = base + (min(rows, r0 + wg_rows) - 1) / a.group;  // position of the last row
  const int b_hi = top < 0 ? 0 : min(top / 64 + 1, kv.width);
  const int low = base + r0 / a.group;
  const int b_lo = a.window > 0 ? max(low - a.window + 1, 0) / 64 : 0;
  const int nb = max(b_hi - b_lo, 0);
  const int per = max((nb + a.splits - 1) / a.splits, wk);
  const int active = max((nb + per - 1) / per, 1);
  if (split >= active) return;
  const int from = b_lo + split * per, to = min(b_hi, from + per);

  // this wave's rows of q, in digits
  i32x4 qd[MR][3][KS];
  float cs[MR];   // factor of the integer scores, without the block's scale
  int pos[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const int row = r0 + (my_r * MR + m) * 16 + c16;
    const bool valid = row < rows;
    pos[m] = valid ? base + row / a.group : -1;
    const float* qp = a.q + (int64_t)(g.t0 + (valid ? row / a.group : 0)) * a.ldq +
                      (int64_t)(g.head * a.group + (valid ? row % a.group : 0)) * dim;
    f32x4 v[KS][4];
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 64 * ks + 16 * g4 + 4 * i;
        v[ks][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (valid && (FULL || d < dim)) v[ks][i] = *reinterpret_cast<const f32x4*>(qp + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          finite = finite && fabsf(v[ks][i][c]) < __builtin_inff();
          amax = fmaxf(amax, fabsf(v[ks][i][c]));
        }
      }
    amax = max4(amax);
    const float bad = add4(finite ? 0.f : 1.f);
    // a row that is not finite gives NaN; one below 1e-30 counts as zero
    // (its scores are, and kTop / amax stays finite)
    const float unit = bad == 0.f && amax > 1e-30f ? kTop / amax : 0.f;
    cs[m] = bad != 0.f ? __builtin_nanf("") : amax / kTop * a.scale;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float f = unit == 0.f ? 0.f : v[ks][i][c] * unit;
          u[c] = (uint32_t)((int)rintf(f) + 0x808080);
        }
        int lo, mid, hi;
        digits4(u, lo, mid, hi);
        qd[m][0][ks][i] = lo;
        qd[m][1][ks][i] = mid;
        qd[m][2][ks][i] = hi;
      }
  }
  const int row_lo = r0 + my_r * MR * 16;
  const int p_lo = base + min(row_lo, rows - 1) / a.group;                  // first row's position
  const int p_hi = base + min(row_lo + MR * 16 - 1, rows - 1) / a.group;    // last row's

  i32x4 zero = {0, 0, 0, 0};
  f32x4 acc[MR][DT];
  float mx[MR], tot[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    mx[m] = kNegInf;
    tot[m] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) acc[m][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t* table = kv.table + (int64_t)g.seq * kv.width;
  const int krow = 16 * (c16 >> 2) + (c16 & 3);  // key of A row c16 in product 0
  int ids = -1;
  for (int i = 0, b = from + my_k; b < to; ++i, b += wk) {
    if ((i & 63) == 0) {  // the next 64 block ids, one a lane
      const int at = b + wk * lane;
      ids = at < to ? table[at] : -1;
    }
    const int id = __builtin_amdgcn_readlane(ids, i & 63);
    if (id < 0 || id >= kv.n_blocks) continue;  // not in the cache: not seen
    const int64_t plane = (int64_t)id * 2 * kv.kvh + g.head;
    const int8_t* kc = kv.codes + plane * (64 * (int64_t)dim);
    const int8_t* vc = kc + (int64_t)kv.kvh * (64 * (int64_t)dim);
    const float dk = kv.scales[plane], dv = kv.scales[plane + kv.kvh];

    i32x4 kf[4][KS], vf[DT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        kf[t][ks] = zero;
        const int d = 64 * ks + 16 * g4;
        if (FULL || d < dim) kf[t][ks] = *reinterpret_cast<const i32x4*>(kc + (krow + 4 * t) * dim + d);
      }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      vf[dt] = zero;
      if (FULL || 16 * dt < dim) vf[dt] = *reinterpret_cast<const i32x4*>(vc + (16 * dt + c16) * 64 + 16 * g4);
    }
    const bool edge = 64 * b + 63 > p_lo || (a.window > 0 && 64 * b <= p_hi - a.window);

#pragma unroll
    for (int m = 0; m < MR; ++m) {
      float s[4][4];
      const float c = cs[m] * dk;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        i32x4 h = zero, l = zero;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          h = mfma(kf[t][ks], qd[m][2][ks], h);
          l = mfma(kf[t][ks], qd[m][1][ks], l);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] <<= 8;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) l = mfma(kf[t][ks], qd[m][0][ks], l);
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][r] = fmaf((float)h[r], 65536.f, (float)l[r]) * c;
      }
      if (edge) {
        const int key = 64 * b + 16 * g4;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = key + 4 * t + r;
            const bool seen = j <= pos[m] && (a.window == 0 || j > pos[m] - a.window);
            s[t][r] = seen ? s[t][r] : kNegInf;
          }
      }
      float bm = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
#pragma unroll
      for (int t = 1; t < 4; ++t)
        bm = fmaxf(bm, fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3])));
      bm = max4(bm);
      const float nm = fmaxf(mx[m], bm);
      const float off = bm == kNegInf ? 0.f : bm;
      const float noff = nm == kNegInf ? 0.f : nm;
      const float alpha = __builtin_amdgcn_exp2f(mx[m] - noff), beta = __builtin_amdgcn_exp2f(bm - noff);
      mx[m] = nm;
      i32x4 ph, pm, pl;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t u[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = __builtin_amdgcn_exp2f(s[t][r] - off);
          sum += p;
          // 2^23 + p kTop, rounded: its low 24 bits are the whole number
          u[r] = __float_as_uint(fmaf(p, kTop, 8388608.f)) + 0x808080u;
        }
        int lo, mid, hi;
        digits4(u, lo, mid, hi);
        pl[t] = lo;
        pm[t] = mid;
        ph[t] = hi;
      }
      tot[m] = fmaf(tot[m], alpha, sum * beta);
      const float f = beta * dv * (1.f / kTop);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        if (!FULL && 16 * dt >= dim) continue;
        const i32x4 h = mfma(vf[dt], ph, zero);
        i32x4 l = mfma(vf[dt], pm, zero);
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] <<= 8;
        l = mfma(vf[dt], pl, l);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[m][dt][r] = fmaf(fmaf((float)h[r], 65536.f, (float)l[r]), f, acc[m][dt][r] * alpha);
      }
    }
  }

  // the waves' sums, row tile by row tile
  const int quads = dim / 4;
  const bool whole = active == 1;
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    if (m > 0) __syncthreads();
    const float t = add4(tot[m]);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      if (FULL || 16 * dt < dim) *reinterpret_cast<f32x4*>(lds + (wave * 16 + c16) * LD + 16 * dt + 4 * g4) = acc[m][dt];
    if (g4 == 0) {
      lds_ml[(wave * 16 + c16) * 2] = mx[m];
      lds_ml[(wave * 16 + c16) * 2 + 1] = t;
    }
    __syncthreads();
    for (int f = threadIdx.x; f < wr * 16 * quads; f += 256) {
      const int lr = f / quads, d = 4 * (f % quads);  // row of the workgroup's wr * 16
      const int w0 = lr >> 4, cr = lr & 15;
      const int row = r0 + (w0 * MR + m) * 16 + cr;
      if (row >= rows) continue;
      float top_m = kNegInf;
      for (int w = w0; w < 4; w += wr) top_m = fmaxf(top_m, lds_ml[(w * 16 + cr) * 2]);
      const float o = top_m == kNegInf ? 0.f : top_m;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      float total = 0.f;
      for (int w = w0; w < 4; w += wr) {
        const float e = __builtin_amdgcn_exp2f(lds_ml[(w * 16 + cr) * 2] - o);
        total = fmaf(lds_ml[(w * 16 + cr) * 2 + 1], e, total);
        const f32x4 p = *reinterpret_cast<const f32x4*>(lds + (w * 16 + cr) * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] = fmaf(p[c], e, sum[c]);
      }
      if (whole) {
        const float inv = total == 0.f ? 0.f : 1.f / total;  // a row that sees nothing is zero
        const float v[4] = {sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv};
        store4(a, g, row, d, v);
      } else {
        const int64_t at = ((int64_t)gid * a.splits + split) * (wg_rows) + (w0 * MR + m) * 16 + cr;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          __hip_atomic_store(a.part + at * dim + d + c, sum[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (d == 0) {
          __hip_atomic_store(a.ml + at * 2, top_m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(a.ml + at * 2 + 1, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
  }
  if (whole) return;

  // Partial sums are device-scope atomic accesses (written through and
  // reloaded by the L2s), so waiting for this lane's own stores before the
  // barrier and the counter's update orders them without a device-scope fence.
  __shared__ int s_last;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&a.cnt[gid], 1) == active - 1;
  __syncthreads();
  if (!s_last) return;
  for (int f = threadIdx.x; f < wg_rows * quads; f += 256) {
    const int lr = f / quads, d = 4 * (f % quads);
    const int row = r0 + lr;
    if (row >= rows) break;
    const int64_t at0 = (int64_t)gid * a.splits * wg_rows + lr;
    float top_m = kNegInf;
    for (int sp = 0; sp < active; ++sp)
      top_m = fmaxf(top_m, __hip_atomic_load(a.ml + (at0 + (int64_t)sp * wg_rows) * 2, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT));
    const float o = top_m == kNegInf ? 0.f : top_m;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
    for (int sp = 0; sp < active; ++sp) {
      const int64_t at = at0 + (int64_t)sp * wg_rows;
      const float e = __builtin_amdgcn_exp2f(
          __hip_atomic_load(a.ml + at * 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) - o);
      total = fmaf(__hip_atomic_load(a.ml + at * 2 + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), e, total);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = fmaf(__hip_atomic_load(a.part + at * dim + d + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), e,
                    v[c]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] *= inv;
    store4(a, g, row, d, v);
  }
  if (threadIdx.x == 0) atomicExch(&a.cnt[gid], 0);
}

AttnPlan attn_plan(int64_t n_seqs, int64_t max_q, int64_t n_heads, int64_t kvh, int64_t dim, int64_t width, int cus) {
  AttnPlan p{};
  const int64_t rows = max_q * (n_heads / kvh);
  p.mr = rows <= 16 ? 1 : 2;
  p.wr = rows <= 16 * p.mr ? 1 : rows <= 32 * p.mr ? 2 : 4;
  const int64_t wg_rows = 16 * p.mr * p.wr;
  p.row_blocks = static_cast<int>((rows + wg_rows - 1) / wg_rows);
  p.groups = n_seqs * kvh * p.row_blocks;
  // two workgroups a compute unit, at least one cache block a wave
  const int64_t most = (width + 4 / p.wr - 1) / (4 / p.wr);
  int64_t s = 2 * (int64_t)cus / p.groups;
  s = s > most ? most : s;
  p.splits = s < 2 ? 1 : static_cast<int>(s);
  if (p.splits > 1) {
    const int64_t sums = p.groups * p.splits * wg_rows;
    p.ws_bytes = kAttnCounterBytes + ((sums * dim * 4 + 255) & ~int64_t(255)) + sums * 8;
  }
  return p;
}

namespace {

template <int KS, int MR, bool FULL>
hipError_t launch_full(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const size_t lds = (4 * 16 * (64 * KS + 4) + 4 * 16 * 2) * sizeof(float);
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_kv_attn<KS, MR, FULL>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_kv_attn<KS, MR, FULL>), dim3((unsigned)(p.groups * a.splits)), dim3(256), lds, st, a);
  return hipGetLastError();
}

template <int KS, int MR>
hipError_t launch(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  return a.kv.dim == 64 * KS ? launch_full<KS, MR, true>(a, p, st) : launch_full<KS, MR, false>(a, p, st);
}

template <int KS>
hipError_t launch_mr(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  return p.mr == 1 ? launch<KS, 1>(a, p, st) : launch<KS, 2>(a, p, st);
}

}  // namespace

hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  switch ((a.kv.dim + 63) / 64) {
    case 1: return launch_mr<1>(a, p, st);
    case 2: return launch_mr<2>(a, p, st);
    case 3: return launch_mr<3>(a, p, st);
    case 4: return launch_mr<4>(a, p, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
