// qmv_attn.hip -- attention of new tokens over the 8-bit block cache, for
// gfx950.
#include "qmv_attn.h"
#include <type_traits>

#include "qmv_device.h"

namespace qmv {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Largest whole number a 24-bit operand holds: 127 * 2^16, so that its three
// base-256 digits all lie within -128..127.
constexpr float kTop = 127 * 65536;
constexpr float kNegInf = -__builtin_inff();
// Units of the weights (kUnit / kTop of what they were chosen by) serve every
// block whose largest weight is up to kAbove bits above it or kBelow below.  They
// are chosen at the first block's own largest weight, later kRoom bits above the
// mean of the blocks so far: each bit of room costs one of the weights', and 0 /
// 1 / 1.5 of them add the sums up in 0.5 / 0.3 / 0.28 of the blocks (16 rows,
// block scales that vary by a factor of two).
constexpr float kAbove = 1.0f, kBelow = 4.0f, kUnit = 2.0f, kRoom = 1.0f;
// Value scales below it count in its units.
constexpr float kTiny = 1e-30f;
// A weight may pass kTop by 32639 units before its top digit turns negative, 0.0056
// bits.  Scores (log2) up to kFar keep that: the largest is rounded where the weight's
// exponent takes it unrounded, by half a step of fp32, and the units' exponent takes
// four more such roundings, together 0.0012 bits.  Beyond kFar a block's scores are
// rounded once, before the maximum is taken from them, so that no exponent lies above
// the maximum's; and the units are chosen at the maximum itself, with no sum to round.
// (The test costs 0 to 1 % of a call's time: 2 x 64 of 16000 96.7 -> 97.6 us, 131072
// tokens unchanged.)
constexpr float kFar = 4096.0f;
// Blocks after which the integer sums are added up at the latest: one adds at
// most 64 * 128 * 127 < 2^20 to a sum.
constexpr int kMost = 1024;

// Waves of a SIMD that the registers leave room for.
constexpr int attn_waves(int dt) { return dt <= 4 ? 3 : dt <= 8 ? 2 : 1; }

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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// a * b rounded to fp32, whatever it is added to.
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// The base-256 digits -128..127 of four whole numbers x: dword e gets digit e
// of all four.  u holds x + 0x8080, or x + 0x808080 where x may be below zero
// (SIGNED), in its low 24 bits: the bytes are then the digits, plus 128 in
// those that the XOR takes it off again.
template <bool SIGNED>
__device__ __forceinline__ void digits4(const uint32_t (&u)[4], int& lo, int& mid, int& hi) {
  const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400);  // u0.b0 u1.b0 u0.b1 u1.b1
  const uint32_t b = __builtin_amdgcn_perm(u[3], u[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0602);  // u0.b2 u1.b2
  const uint32_t e = __builtin_amdgcn_perm(u[3], u[2], 0x06020c0c);
  lo = (int)(__builtin_amdgcn_perm(b, a, 0x05040100) ^ 0x80808080u);
  mid = (int)(__builtin_amdgcn_perm(b, a, 0x07060302) ^ 0x80808080u);
  hi = (int)(SIGNED ? (c | e) ^ 0x80808080u : c | e);
}

__device__ __forceinline__ float wave_max(float v) {
  v = max8(v);
  v = fmaxf(v, dpp_f<DPP_MIRROR>(v));
  const int b = __float_as_int(v);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}

// A value that all lanes have, in a scalar register.
__device__ __forceinline__ float scalar(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }

// Two floats at once, device scope.
__device__ __forceinline__ void store8(float* p, float x, float y) {
  const uint64_t v = ((uint64_t)__float_as_uint(y) << 32) | __float_as_uint(x);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void load8(const float* p, float& x, float& y) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  x = __uint_as_float((uint32_t)v);
  y = __uint_as_float((uint32_t)(v >> 32));
}

// 16 cached bytes of a lane.  Where no other wave reads them they pass the
// caches by.
template <bool ONCE>
__device__ __forceinline__ i32x4 load_codes(const int8_t* p) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p));
  else
    return *reinterpret_cast<const i32x4*>(p);
}

// The rows of one (sequence, kv head, row block) and the share of its cache
// blocks that a workgroup takes.
struct Group {
  int seq, head, rb;   // sequence, kv head, row block
  int t0, n, len;      // first row, new tokens, length
  int splits, split;   // workgroups that may share it, and which this is
  int slot;            // the first one's slot in the workspace
};

// Rows of a sequence, clamped to what the call has.
__device__ __forceinline__ void rows_of(const KvView& kv, int seq, int& t0, int& n, int& len) {
  t0 = seq * kv.max_q;
  n = kv.max_q;
  if (kv.start != nullptr) {
    t0 = min(max(kv.start[seq], 0), kv.n_tok);
    n = min(max(kv.start[seq + 1], t0), kv.n_tok) - t0;
    n = min(n, kv.max_q);
  }
  len = max(kv.lens[seq], 0);
}

// Cache blocks [lo, hi) that the rows at positions first .. last see.
__device__ __forceinline__ void blocks_of(const AttnArgs& a, int first, int last, int& lo, int& hi) {
  hi = last < 0 ? 0 : min(last / 64 + 1, a.kv.width);
  lo = a.window > 0 ? max(max(first, 0) - a.window + 1, 0) / 64 : 0;  // positions below zero see nothing
}

__device__ __forceinline__ int wave_add(int v) {
  v = sum8(v);
  v += dpp_i<DPP_MIRROR>(v);
  return (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
         (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
}

// With a.shares (at most 64 sequences, no more groups than a.shares) sequences
// are split by their lengths: a lane takes a sequence, and the workgroups of a
// group are as many as parts of at most q cache blocks need, q the smallest of
// a geometric series for which all parts are at most a.shares.
struct Lengths {
  int t0, n, len;       // of this lane's sequence
  int parts, rbs, end;  // workgroups of a group, row blocks, where its last group's workgroups end
};

__device__ __forceinline__ Lengths lengths_of(const AttnArgs& a, int wg_rows, int wk) {
  const int lane = threadIdx.x & 63;
  Lengths s{};
  int run = 0;
  if (lane < a.kv.n_seqs) {
    rows_of(a.kv, lane, s.t0, s.n, s.len);
    int lo, hi;
    blocks_of(a, s.len - s.n, s.len - 1, lo, hi);
    run = max(hi - lo, 1);
  }
  s.rbs = (s.n * a.group + wg_rows - 1) / wg_rows;  // 0 without rows
  const int times = a.kv.kvh * s.rbs;
  int q = max((wave_add(run * times) + a.shares - 1) / a.shares, wk);
  q = max(q, a.least);
  // A run of up to two blocks a wave has one part.  No lane may leave the loop
  // or take another way through it than the others: wave_add reads them all.
  // (So no condition on run inside it, which the compiler made two loops of,
  // the second without the lanes that the sum is read from; and a bound that
  // q, which passes any run long before it, cannot reach.)
  const int whole = run <= 2 * wk ? max(run, 1) : 1;
  s.parts = 0;
  for (int i = 0; i < 256; ++i) {
    const int each = max(q, whole);
    s.parts = (run + each - 1) / each;
    if (wave_add(s.parts * times) <= a.shares) break;
    q += q / 8 + 1;
  }
  s.end = s.parts * times;
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const int y = __shfl_up(s.end, k, 64);
    if (lane >= k) s.end += y;
  }
  return s;
}

__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The device hands workgroup w to XCD w % 8.  This order gives each XCD, which
// has an L2 of its own, neighbouring ones: the row blocks that read the same
// cache blocks (us without / with: a prompt of 2048, 8 heads with 4 query heads,
// 128 dims 173 / 145, 2 x 64 new tokens of 16000 98.7 / 96.7, 8 x 9 of 5001 with
// 16 query heads 128.8 / 130.7).
__device__ __forceinline__ int near_order(int w, int n) {
  const int xcd = w & 7, at = w >> 3;
  return xcd * (n >> 3) + min(xcd, n & 7) + at;
}

// What workgroup w does; false: nothing.  Without a.shares every group has
// a.splits workgroups.
__device__ __forceinline__ bool group_of(const AttnArgs& a, int w, int wg_rows, int wk, Group& g) {
  if (a.shares == 0) {
    const int gid = w / a.splits;
    g.split = w - gid * a.splits;
    g.splits = a.splits;
    g.slot = gid * a.splits;
    g.rb = gid % a.row_blocks;
    g.head = gid / a.row_blocks % a.kv.kvh;
    g.seq = gid / a.row_blocks / a.kv.kvh;
    rows_of(a.kv, g.seq, g.t0, g.n, g.len);
    return true;
  }
  const Lengths s = lengths_of(a, wg_rows, wk);
  const uint64_t hit = __ballot(w < s.end);  // the sequences that end behind w
  if (hit == 0) return false;
  g.seq = __builtin_ctzll(hit);
  g.t0 = lane_of(s.t0, g.seq);
  g.n = lane_of(s.n, g.seq);
  g.len = lane_of(s.len, g.seq);
  g.splits = lane_of(s.parts, g.seq);
  const int rbs = lane_of(s.rbs, g.seq);
  const int rel = w - (lane_of(s.end, g.seq) - g.splits * a.kv.kvh * rbs), i = rel / g.splits;
  g.split = rel - i * g.splits;
  g.slot = w - g.split;
  g.head = i / rbs;
  g.rb = i - g.head * rbs;
  return true;
}

// Cache blocks [lo, hi) of a group, and how many of its workgroups have a
// share of them, `per` blocks each; false: it has no rows.
__device__ __forceinline__ bool blocks_of(const AttnArgs& a, const Group& g, int wg_rows, int wk, int& lo, int& hi,
                                          int& per, int& active) {
  const int rows = g.n * a.group, r0 = g.rb * wg_rows, base = g.len - g.n;
  if (r0 >= rows) return false;
  blocks_of(a, base + r0 / a.group, base + (min(rows, r0 + wg_rows) - 1) / a.group, lo, hi);
  const int nb = max(hi - lo, 0);
  per = max((nb + g.splits - 1) / g.splits, wk);
  active = max((nb + per - 1) / per, 1);
  return true;
}

// Factors of the n parts of row lr of a group, one part a lane (at most 64).
__device__ __forceinline__ float factor_of(const AttnArgs& a, int64_t slot, int wg_rows, int lr, int n) {
  const int lane = threadIdx.x & 63;
  float m, l;
  load8(a.ml + ((slot + min(lane, n - 1)) * wg_rows + lr) * 2, m, l);
  m = lane < n ? m : kNegInf;
  l = lane < n ? l : 0.f;
  const float top = wave_max(m);
  const float e = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m - top);
  const float sum = wave_sum(l * e);
  return sum == 0.f ? 0.f : e / sum;
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
// operand of each product is a whole number of 24 bits, as three base-256
// digits: a row of q in units of its largest value / kTop, the weights P dv in
// units that follow the row's largest (below).  A product is then three exact
// integer products, whose sums meet in fp32; no code is ever converted.
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
// The three integer sums of O stay in the matrix registers from block to
// block, as long as every row's largest weight in the block lies within
// 2^-kBelow .. 2^kAbove of what the units were chosen by; else they are added
// to the fp32 sums in LDS (280 instructions at 96 dims, against 250 of a block)
// and the units chosen anew.  A weight is so rounded to half a unit, at most
// 16 / kTop (just above 2^-19) of the largest of its block, mostly 2^-22, and a block costs the vector ALU
// nothing for O (KEEP; above 128 dims the integer sums do not fit the
// registers, and fp32 sums take a block's products: 160 of 380 instructions at
// 128 dims).
//
// A wave owns 16 rows; of a workgroup's NW waves WR lie along the rows (ONE:
// one does) and NW / WR along the cache blocks, and several workgroups share
// a group's blocks (group_of).  K of the next block is loaded when the scores
// of this one are done, V when its product is: the loads need no registers of
// their own and have half a block's work to arrive in.  q's digits are made
// once a workgroup, through LDS.  The waves' sums meet in LDS in wave order, the
// workgroups' through the workspace: the last one to arrive (up to 16 rows, ONE)
// or a launch of its own (k_kv_join) adds them in split order, so the result does
// not depend on timing.  DT: 16-dim tiles of the head dimension.
//
// Bound by the cache's bytes where a wave's rows are few: 131072 tokens, 8
// heads, 128 dims in 52.6 us, of which 40 stream the cache at 6.7 TB/s and the
// rest is the start (ids, then blocks, then q: 3 us), the waves' unequal ends
// (5), the joins (4) and the launch.  48 sequences of up to 12000: 122 us, 4.8
// TB/s.  With many rows by waiting for blocks that the waves along the rows and
// the row blocks read again from L2 (a third of the waves' time; 2 x 64 new
// tokens of 16000, 5 x 8 heads, 96 dims: 97 us, of them 52 vector ALU, 22 matrix
// ALU).  Through LDS once a workgroup they cost more: waves in step do not
// overlap one's products with another's exponentials (120 to 152 us).
template <int DT, int NW, int WR>
__global__ __launch_bounds__(64 * NW, attn_waves(DT)) void k_kv_attn(AttnArgs a) {
  constexpr bool KEEP = DT <= 8;
  constexpr bool ONE = WR == 1;
  constexpr int KS = (DT + 3) / 4;     // 64-value steps of a score
  constexpr int LD = 16 * DT + 4;      // LDS row stride of the sums (floats)
  constexpr int QLD = 64 * KS + 16;    // and of q's digits (bytes)
  constexpr int T = 64 * NW;
  constexpr bool QREG = KS <= 2;       // q's digits stay in registers
  extern __shared__ __align__(16) float lds[];       // [NW][16 rows][LD] fp32 sums, [NW][16][2] (maximum, total), digits of q
  float* lds_ml = lds + NW * 16 * LD;
  int8_t* lds_q = reinterpret_cast<int8_t*>(lds_ml + NW * 16 * 2);  // [3][16 wr][QLD]
  __shared__ float s_unit[16 * NW];
  const KvView& kv = a.kv;
  constexpr int dim = 16 * DT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g4 = lane >> 4;
  constexpr int wr = WR, wk = NW / WR, wg_rows = 16 * WR;
  const int my_r = wave % wr, my_k = wave / wr;
  Group g;
  if (!group_of(a, a.row_blocks > 1 ? near_order(blockIdx.x, gridDim.x) : blockIdx.x, wg_rows, wk, g)) return;
  int b_lo, b_hi, per, active;
  if (!blocks_of(a, g, wg_rows, wk, b_lo, b_hi, per, active)) return;
  if (g.split >= active) return;
  const int rows = g.n * a.group;
  const int r0 = g.rb * wg_rows;
  const int base = g.len - g.n;  // position of the sequence's first new token
  const int from = b_lo + g.split * per, to = min(b_hi, from + per);

  // q: 16 lanes a row, four rows a wave at a time
  constexpr int QJ = 4 * WR > NW ? 4 * WR / NW : 1;  // passes
  const int n_rows = min(rows - r0, wg_rows);
  f32x4 qv[QJ][KS];
#pragma unroll
  for (int j = 0; j < QJ; ++j) {
    const int lr = (j * NW + wave) * 4 + g4;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qv[j][ks] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int d = 64 * ks + 4 * c16;
      if (lr < n_rows && d < dim) {
        const int row = r0 + lr;
        qv[j][ks] = *reinterpret_cast<const f32x4*>(a.q + (int64_t)(g.t0 + row / a.group) * a.ldq +
                                                   (int64_t)(g.head * a.group + row % a.group) * dim + d);
      }
    }
  }

  const i32x4 zero = {0, 0, 0, 0};
  const int krow = 16 * (c16 >> 2) + (c16 & 3);  // key of A row c16 in product 0
  const int voff = c16 * 64 + 16 * g4;
  i32x4 kf[4][KS], vf[DT];
  // Past the head dimension q's digits are zero, whatever K's are: such lanes
  // read bytes that others read too.
  auto load_k = [&](int64_t plane) {
    const int8_t* kc = kv.codes + plane * (64 * (int64_t)dim);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int d = DT % 4 == 0 ? 64 * ks + 16 * g4 : min(64 * ks + 16 * g4, dim - 16);
        kf[t][ks] = load_codes<ONE>(kc + (uint32_t)((krow + 4 * t) * dim + d));
      }
  };
  auto load_v = [&](int64_t plane) {
    const int8_t* vc = kv.codes + (plane + kv.kvh) * (64 * (int64_t)dim);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) vf[dt] = load_codes<ONE>(vc + (uint32_t)(voff + 1024 * dt));
  };
  // Ids and scales of 64 blocks at a time, one a lane; blocks that are not in
  // the cache are left out.  todo: the lanes whose blocks are still to be
  // loaded, cur the one that is in the registers.
  const int32_t* table = kv.table + (int64_t)g.seq * kv.width;
  int c0 = from + my_k - 64 * wk, ids = -1, cur = 0;
  float dks = 0.f, dvs = 0.f;
  uint64_t todo = 0;
  int64_t plane = 0;
  auto take = [&]() {
    cur = __builtin_ctzll(todo);
    todo &= todo - 1;
    plane = (int64_t)__builtin_amdgcn_readlane(ids, cur) * 2 * kv.kvh + g.head;
  };
  auto open = [&]() -> bool {
    for (c0 += 64 * wk; c0 < to; c0 += 64 * wk) {
      const int at = c0 + wk * lane;
      ids = at < to ? table[at] : -1;
      const bool in = ids >= 0 && ids < kv.n_blocks;
      const float* sp = kv.scales + (in ? (int64_t)ids * 2 * kv.kvh + g.head : 0);
      dks = in ? sp[0] : 0.f;
      dvs = in ? sp[kv.kvh] : 0.f;
      todo = __ballot(in);
      if (todo == 0) continue;
      take();
      load_k(plane);
      load_v(plane);
      return true;
    }
    return false;
  };
  bool more = open();

  // q in digits, while the first block arrives.  A row below 1e-30 counts as
  // zero (its scores are, and kTop / amax stays finite), as does one that is
  // not finite, whose total becomes NaN; the sign of the scale is q's, so that
  // factors of the integer scores are not below zero.
#pragma unroll
  for (int j = 0; j < QJ; ++j) {
    const int lr = (j * NW + wave) * 4 + g4;
    float amax = 0.f, odd = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        amax = fmaxf(amax, fabsf(qv[j][ks][c]));
        odd += qv[j][ks][c] * 0.f;  // NaN if it is not finite
      }
    amax = max8(amax);
    amax = fmaxf(amax, dpp_f<DPP_MIRROR>(amax));
    odd = sum8(odd);
    odd += dpp_f<DPP_MIRROR>(odd);
    float unit = odd == 0.f && amax > 1e-30f ? kTop / amax : 0.f;
    if (a.scale < 0.f) unit = -unit;
    if (c16 == 0 && lr < wg_rows) s_unit[lr] = odd == 0.f ? (unit == 0.f ? 0.f : amax / kTop * fabsf(a.scale)) : odd;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float f = unit == 0.f ? 0.f : qv[j][ks][c] * unit;
        u[c] = (uint32_t)((int)rintf(f) + 0x808080);
      }
      int x[3];
      digits4<true>(u, x[0], x[1], x[2]);
      if (lr < wg_rows)
#pragma unroll
        for (int e = 0; e < 3; ++e)
          *reinterpret_cast<int*>(lds_q + (e * wg_rows + lr) * QLD + 64 * ks + 4 * c16) = x[e];
    }
  }
  __syncthreads();
  const int8_t* my_q = lds_q + (my_r * 16 + c16) * QLD + 16 * g4;
  auto q_of = [&](int e, int ks) {
    return *reinterpret_cast<const i32x4*>(my_q + e * wg_rows * QLD + 64 * ks);
  };
  i32x4 qd[3][QREG ? KS : 1];
  if constexpr (QREG)
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qd[e][ks] = q_of(e, ks);
  const float cs = s_unit[my_r * 16 + c16];  // factor of the integer scores, without the block's; NaN: the row is
  const float csf = cs == cs ? cs : 0.f;
  const int row = r0 + my_r * 16 + c16;
  const int pos = row < rows ? max(base + row / a.group, -1) : -1;
  const int row_lo = r0 + my_r * 16;
  const int p_lo = base + min(row_lo, rows - 1) / a.group;        // first row's position
  const int p_hi = max(base + min(row_lo + 15, rows - 1) / a.group, -1);  // last row's

  // sums of O^T: fp32, or (KEEP) one integer sum a digit, fp32 ones in LDS
  constexpr int NI = KEEP ? DT : 1, NF = KEEP ? 1 : DT;
  i32x4 oh[NI], om[NI], ol[NI];
  f32x4 of[NF];
  float mx = kNegInf, total = 0.f;  // of the fp32 sums: what weights are relative to (log2), and their total
  float ref = kNegInf, tot = 0.f;   // the same of the integer sums
  float dref = 1.f, lref = 0.f, per_dref = kTop / kUnit;  // value scale that the units were chosen by
  int since = 0;                    // blocks in the integer sums
  bool fresh = true;                // nothing is in the fp32 sums
  float mean = kNegInf;             // of the blocks' largest weights times value scale (log2), the last ones count most
  float* mine = lds + (wave * 16 + c16) * LD + 4 * g4;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
    if constexpr (KEEP)
      oh[dt] = om[dt] = ol[dt] = zero;
    else
      of[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // the integer sums into the fp32 ones
  auto add_up = [&]() {
    const float nm = fmaxf(mx, ref);
    const float keep = mx == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mx - nm);
    const float w = ref == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ref - nm);
    const float f = w * (dref * (kUnit / kTop));
    if constexpr (KEEP) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        f32x4* at = reinterpret_cast<f32x4*>(mine + 16 * dt);
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if (!fresh) s = *at;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = fmaf((float)oh[dt][r], 65536.f, fmaf((float)om[dt][r], 256.f, (float)ol[dt][r]));
          s[r] = fmaf(x, f, s[r] * keep);
        }
        *at = s;
        oh[dt] = om[dt] = ol[dt] = zero;
      }
    }
    total = fmaf(total, keep, tot * w);
    tot = 0.f;
    mx = nm;
    since = 0;
    fresh = false;
  };

  while (more) {
    const int b = c0 + wk * cur;
    const float dk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dks), cur));
    const float dv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dvs), cur));
    float s[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      i32x4 h = zero, l = zero;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        l = mfma(kf[t][ks], QREG ? qd[1][QREG ? ks : 0] : q_of(1, ks), l);
        h = mfma(kf[t][ks], QREG ? qd[2][QREG ? ks : 0] : q_of(2, ks), h);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) l[r] <<= 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) l = mfma(kf[t][ks], QREG ? qd[0][QREG ? ks : 0] : q_of(0, ks), l);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] = fmaf((float)h[r], 65536.f, (float)l[r]);
    }
    const bool next = todo != 0;
    if (next) {
      take();
      load_k(plane);
    }
    float c = csf * dk;
    if (64 * b + 63 > p_lo || (a.window > 0 && 64 * b <= p_hi - a.window)) {
      const int key = 64 * b + 16 * g4;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = key + 4 * t + r;
          const bool seen = j <= pos && (a.window == 0 || j > pos - a.window);
          s[t][r] = seen ? s[t][r] * c : kNegInf;
        }
      c = 1.f;
    }
    float bm = max3(s[0][0], s[0][1], s[0][2]);
#pragma unroll
    for (int i = 3; i < 15; i += 2) bm = max3(bm, s[i / 4][i % 4], s[(i + 1) / 4][(i + 1) % 4]);
    bm = fmaxf(bm, s[3][3]);
    bm = product(max4(bm), c);
    const bool some_far =
        (__builtin_amdgcn_ballot_w64(bm > kNegInf) & __builtin_amdgcn_ballot_w64(fabsf(bm) > kFar)) != 0;
    if (some_far) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][r] = product(s[t][r], c);
      c = 1.f;
    }
    if constexpr (KEEP) {
      // x: log2 of the largest weight times value scale over what the units were
      // chosen by.  They follow the mean of the blocks so far.
      const float dvu = fmaxf(dv, kTiny);
      const float lr = dv > 0.f ? __builtin_amdgcn_logf(dvu) - lref : 0.f;
      const float rel = bm - ref, x = rel + lr;
      const bool any = bm > kNegInf, anew = any && !(x <= kAbove && x >= -kBelow && rel <= 30.f);
      const float top = bm + lr + lref;
      mean = !any ? mean : mean == kNegInf ? top : fmaf(top - mean, 0.125f, mean);
      if (__any(anew) || since >= kMost) {
        if (since > 0) add_up();
        if (fabsf(lr) > 8.f || (some_far && lr != 0.f)) {  // units by this block's value scale
          dref = scalar(dvu);
          lref = scalar(lref + lr);
          per_dref = scalar(kTop / kUnit / dvu);
        }
        const float r = fminf(fmaxf(mean + (ref == kNegInf ? 0.f : kRoom), top - kAbove), top + kBelow) - lref;
        ref = any ? (fabsf(bm) > kFar ? bm : r) : ref;
      }
    } else {
      ref = bm;
      dref = dv > 0.f ? dv : 1.f;
    }
    const float cw = KEEP ? dv * per_dref : dv / dref * (kTop / kUnit);
    const float off = ref == kNegInf ? 0.f : ref;
    i32x4 ph, pm, pl;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t u[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -off));
        sum += p;
        // 2^23 + 0x8080 + the whole number, rounded, in the low 24 bits
        u[r] = __float_as_uint(fmaf(p, cw, 8388608.f + 32896.f));
      }
      int lo, mid, hi;
      digits4<false>(u, lo, mid, hi);
      pl[t] = lo;
      pm[t] = mid;
      ph[t] = hi;
    }
    if constexpr (KEEP) {
      tot += sum;
      ++since;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        oh[dt] = mfma(vf[dt], ph, oh[dt]);
        om[dt] = mfma(vf[dt], pm, om[dt]);
        ol[dt] = mfma(vf[dt], pl, ol[dt]);
      }
    } else {
      const float nm = fmaxf(mx, bm);
      const float keep = mx == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mx - nm);
      const float w = bm == kNegInf ? 0.f : __builtin_amdgcn_exp2f(bm - nm);
      const float f = w * (dref * (kUnit / kTop));
      total = fmaf(total, keep, sum * w);
      mx = nm;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const i32x4 h = mfma(vf[dt], ph, zero);
        i32x4 l = mfma(vf[dt], pm, zero);
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] <<= 8;
        l = mfma(vf[dt], pl, l);
#pragma unroll
        for (int r = 0; r < 4; ++r) of[dt][r] = fmaf(fmaf((float)h[r], 65536.f, (float)l[r]), f, of[dt][r] * keep);
      }
    }
    if (next)
      load_v(plane);
    else
      more = open();
  }
  if constexpr (KEEP) {
    if (since > 0 || fresh) add_up();
  } else {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<f32x4*>(mine + 16 * dt) = of[dt];
  }

  // the waves' sums, then the workgroups'
  total = add4(total);
  if (g4 == 0) {
    lds_ml[(wave * 16 + c16) * 2] = mx;
    lds_ml[(wave * 16 + c16) * 2 + 1] = cs != cs && total > 0.f ? cs : total;
  }
  __syncthreads();
  const int quads = dim / 4;
  const bool whole = active == 1;
  for (int f = threadIdx.x; f < n_rows * quads; f += T) {
    const int lr = f / quads, d = 4 * (f % quads);  // row of the workgroup
    const int w0 = lr / 16, tr = lr % 16;
    float top_m = kNegInf;
    for (int w = w0; w < NW; w += wr) top_m = fmaxf(top_m, lds_ml[(w * 16 + tr) * 2]);
    const float o = top_m == kNegInf ? 0.f : top_m;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    for (int w = w0; w < NW; w += wr) {
      const float e = __builtin_amdgcn_exp2f(lds_ml[(w * 16 + tr) * 2] - o);
      sum = fmaf(lds_ml[(w * 16 + tr) * 2 + 1], e, sum);
      const f32x4 x = *reinterpret_cast<const f32x4*>(lds + (w * 16 + tr) * LD + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(x[i], e, v[i]);
    }
    if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing is zero
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= inv;
      store4(a, g, r0 + lr, d, v);
    } else {
      const int64_t at = (int64_t)(g.slot + g.split) * wg_rows + lr;
      if constexpr (!ONE) {
        *reinterpret_cast<f32x4*>(a.part + at * dim + d) = f32x4{v[0], v[1], v[2], v[3]};
      } else {
        store8(a.part + at * dim + d, v[0], v[1]);
        store8(a.part + at * dim + d + 2, v[2], v[3]);
      }
      if (d == 0) store8(a.ml + at * 2, top_m, sum);
    }
  }
  if constexpr (!ONE) return;  // k_kv_join
  if (whole) return;

  // Partial sums are device-scope atomic accesses (written through and
  // reloaded by the L2s), so waiting for this lane's own stores before the
  // barrier and the counter's update orders them without a device-scope fence.
  __shared__ int s_last;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&a.cnt[g.slot], 1) == active - 1;
  __syncthreads();
  if (!s_last) return;
  const int64_t at0 = (int64_t)g.slot * wg_rows;
  for (int lr = wave; lr < n_rows; lr += NW) {
    const float f = factor_of(a, g.slot, wg_rows, lr, active);
    if (lane < active) lds[lr * active + lane] = f;
  }
  if (threadIdx.x == 0) atomicExch(&a.cnt[g.slot], 0);
  __syncthreads();
  const int items = n_rows * quads;
  // with few outputs, several threads share one along the splits
  const int sub = items >= T ? 1 : T / items;
  const int share = (active + sub - 1) / sub;
  float* meet = lds + ((n_rows * active + 3) & ~3);  // 16-byte accesses
  for (int f0 = 0; f0 < items; f0 += T) {
    const int f = sub == 1 ? f0 + (int)threadIdx.x : (int)threadIdx.x % items;
    const int part = sub == 1 ? 0 : (int)threadIdx.x / items;
    const int lr = f / quads, d = 4 * (f % quads);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (f < items && part < sub) {
      const int s1 = min(active, (part + 1) * share);
      const float* src = a.part + (at0 + lr) * dim + d;
      auto add = [&](int sp, auto batch) {  // so many at once
        constexpr int B = decltype(batch)::value;
        float x[B][4];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const int64_t k = (int64_t)min(sp + j, s1 - 1) * wg_rows * dim;
          load8(src + k, x[j][0], x[j][1]);
          load8(src + k + 2, x[j][2], x[j][3]);
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const float e = sp + j < s1 ? lds[lr * active + sp + j] : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = fmaf(x[j][i], e, v[i]);
        }
      };
      int sp = part * share;
      for (; sp + 4 < s1; sp += 16) add(sp, std::integral_constant<int, 16>());
      if (sp < s1) add(sp, std::integral_constant<int, 4>());
    }
    if (sub > 1) {
      if (part > 0 && part < sub) *reinterpret_cast<f32x4*>(meet + ((part - 1) * items + f) * 4) = f32x4{v[0], v[1], v[2], v[3]};
      __syncthreads();
      if (part > 0) return;
      for (int p = 1; p < sub; ++p) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(meet + ((p - 1) * items + f) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[i];
      }
    }
    if (f < items) store4(a, g, r0 + lr, d, v);
  }
}

// The join of groups of more than 16 rows, as a launch of its own over all of
// the device: a workgroup alone reads partial sums at some 60 GB/s (8 heads, 64
// rows each, 128 dims, us joined by the last workgroup / by this: 700 tokens
// 25.7 / 16.1, 8000 tokens 39.8 / 23.0; 8 rows and 131072 tokens 52.7 / 53.8,
// 48 sequences of up to 12000 122 / 129).  A thread joins four values of a row,
// `chunks` workgroups a group; bound by the launch and two loads in a row.
__global__ __launch_bounds__(256) void k_kv_join(AttnArgs a, int wg_rows, int wk, int chunks) {
  __shared__ float fac[66 * kAttnMaxSplits];  // rows of 256 threads, at least four threads a row
  const int gid = blockIdx.x / chunks, chunk = blockIdx.x - gid * chunks;
  Group g;
  g.rb = gid % a.row_blocks;
  g.head = gid / a.row_blocks % a.kv.kvh;
  g.seq = gid / a.row_blocks / a.kv.kvh;
  rows_of(a.kv, g.seq, g.t0, g.n, g.len);
  g.splits = a.splits;
  g.slot = gid * a.splits;
  if (a.shares > 0) {
    const Lengths s = lengths_of(a, wg_rows, wk);
    const int rbs = lane_of(s.rbs, g.seq);
    g.splits = lane_of(s.parts, g.seq);
    g.slot = lane_of(s.end, g.seq) - g.splits * (a.kv.kvh * rbs - g.head * rbs - g.rb);
  }
  int lo, hi, per, active;
  if (!blocks_of(a, g, wg_rows, wk, lo, hi, per, active) || active == 1) return;
  const int r0 = g.rb * wg_rows, n_rows = min(g.n * a.group - r0, wg_rows);
  const int quads = a.kv.dim / 4, items = n_rows * quads, f0 = chunk * 256;
  if (f0 >= items) return;
  const int lr0 = f0 / quads, lr1 = min(n_rows, (f0 + 255) / quads + 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int lr = lr0 + wave; lr < lr1; lr += 4) {
    const float f = factor_of(a, g.slot, wg_rows, lr, active);
    if (lane < active) fac[(lr - lr0) * active + lane] = f;
  }
  __syncthreads();
  const int f = f0 + (int)threadIdx.x;
  if (f >= items) return;
  const int lr = f / quads, d = 4 * (f % quads);
  const float* src = a.part + ((int64_t)g.slot * wg_rows + lr) * a.kv.dim + d;
  const float* fs = fac + (lr - lr0) * active;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int B = 16;  // so many at once
  for (int sp = 0; sp < active; sp += B) {
    f32x4 x[B];
#pragma unroll
    for (int j = 0; j < B; ++j)
      x[j] = *reinterpret_cast<const f32x4*>(src + (int64_t)min(sp + j, active - 1) * wg_rows * a.kv.dim);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const float e = sp + j < active ? fs[sp + j] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(x[j][i], e, v[i]);
    }
  }
  store4(a, g, r0 + lr, d, v);
}

AttnPlan attn_plan(int64_t n_seqs, int64_t max_q, int64_t n_heads, int64_t kvh, int64_t dim, int64_t width, int cus) {
  AttnPlan p{};
  const int64_t rows = max_q * (n_heads / kvh), tiles = (rows + 15) / 16;
  // Workgroups of eight waves make fewer partial sums of one sequence, those of
  // four are more alike in length where sequences share the device (us, four /
  // eight waves, 128 dims: one sequence of 131072 tokens and eight heads 57.0 /
  // 53.5, of 700 12.9 / 11.1; 48 of up to 12000 126 / 153, 16 of up to 8000
  // 37.7 / 41.1).
  const bool small = dim <= 128;
  const int64_t all = n_seqs * kvh * tiles;
  p.nw = small && (all <= (tiles > 1 ? cus : cus / 4) || tiles >= 4) ? 8 : 4;
  // Rows beyond 16: waves along the rows share a cache block's way from L2, those
  // along the blocks make runs shorter, which counts while the device is not full
  // of row tiles (us, at most two / four waves along the rows, 128 dims, 8 heads
  // with 8 query heads: one sequence of 8000 with 8 new tokens 19.8 / 22.9, four
  // with 16 60.8 / 62.6; 16 of 4000 with 8 77.1 / 67.0).
  p.wr = 1;
  while (p.wr < (all <= cus ? 2 : 4) && p.wr < tiles) p.wr *= 2;
  const int64_t wg_rows = 16 * p.wr, wk = p.nw / p.wr;
  p.row_blocks = static_cast<int>((rows + wg_rows - 1) / wg_rows);
  p.groups = n_seqs * kvh * p.row_blocks;
  // Workgroups that the device holds at once: their registers leave room for
  // eight waves a compute unit, four above 128 dims.  More at a time would
  // start one after the other, each with its own start and end.
  const int64_t slots = (int64_t)cus * (small ? 8 : 4) / p.nw;
  // Up to two cache blocks a wave are not shared, which costs a join through
  // the workspace; more are, down to one a wave (one sequence, eight heads, us
  // against at least two a wave: 700 tokens 11.2 unshared, 12.0 shared; 2000
  // tokens 12.7 / 15.6, 8192 14.4 / 18.2).
  const int64_t most = width <= 2 * wk ? 1 : (width + wk - 1) / wk;
  int64_t s = slots / p.groups;
  s = s > most ? most : s;
  s = s > kAttnMaxSplits ? kAttnMaxSplits : s;
  p.splits = s < 2 ? 1 : static_cast<int>(s);
  p.grid = p.groups * p.splits;
  p.least = static_cast<int>((width + kAttnMaxSplits - 1) / kAttnMaxSplits);
  // where a join is a launch of its own, only if every group could have two
  // parts (8 sequences of 1000, 128 new tokens, 64 dims: 41.1 us against 47.9)
  if (n_seqs > 1 && n_seqs <= 64 && most > 1 && p.groups <= (p.wr > 1 ? slots : 2 * slots)) {
    // twice the slots where there are nearly as many groups already (64
    // sequences of up to 8000 tokens, eight heads: 117 us against 129)
    p.shares = static_cast<int>(5 * p.groups <= 4 * slots ? slots : 2 * slots);
    p.grid = p.shares;
  }
  if (p.splits > 1 || p.shares > 0) {
    const int64_t sums = p.grid * wg_rows;
    p.ws_bytes = kAttnCounterBytes + ((sums * dim * 4 + 255) & ~int64_t(255)) + sums * 8;
  }
  return p;
}

namespace {

template <int DT, int NW, int WR>
hipError_t launch_one(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  constexpr int lds = NW * 16 * ((16 * DT + 4) + 2) * 4 + 3 * 16 * WR * (64 * ((DT + 3) / 4) + 16);
  // the join's factors, and the sums that meet (WR 1)
  static_assert(WR > 1 || lds >= (16 * kAttnMaxSplits + 4 * 64 * NW) * 4);
  if (lds > 60 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_kv_attn<DT, NW, WR>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_kv_attn<DT, NW, WR>), dim3((unsigned)(a.part != nullptr ? p.grid : p.groups)), dim3(64 * NW),
                     lds, st, a);
  return hipGetLastError();
}

template <int DT, int NW>
hipError_t launch_rows(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (p.wr == 1) return launch_one<DT, NW, 1>(a, p, st);
  if (p.wr == 2) return launch_one<DT, NW, 2>(a, p, st);
  return launch_one<DT, NW, 4>(a, p, st);
}

template <int DT>
hipError_t launch(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if constexpr (DT <= 8)
    if (p.nw == 8) return launch_rows<DT, 8>(a, p, st);
  return launch_rows<DT, 4>(a, p, st);
}

// Every multiple of 16 dims has its own kernel: one for the next multiple of 32
// or 64, with a bound on its tiles, spilled registers (8 x 8 new tokens of
// 8000, 160 dims: 138 us, 86 with its own).
hipError_t launch_sums(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  switch (a.kv.dim / 16) {
    case 1: return launch<1>(a, p, st);
    case 2: return launch<2>(a, p, st);
    case 3: return launch<3>(a, p, st);
    case 4: return launch<4>(a, p, st);
    case 5: return launch<5>(a, p, st);
    case 6: return launch<6>(a, p, st);
    case 7: return launch<7>(a, p, st);
    case 8: return launch<8>(a, p, st);
    case 9: return launch<9>(a, p, st);
    case 10: return launch<10>(a, p, st);
    case 11: return launch<11>(a, p, st);
    case 12: return launch<12>(a, p, st);
    case 13: return launch<13>(a, p, st);
    case 14: return launch<14>(a, p, st);
    case 15: return launch<15>(a, p, st);
    case 16: return launch<16>(a, p, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const hipError_t e = launch_sums(a, p, st);
  if (e != hipSuccess || a.part == nullptr || p.wr == 1) return e;
  const int wg_rows = 16 * p.wr, chunks = (wg_rows * (a.kv.dim / 4) + 255) / 256;
  hipLaunchKernelGGL(k_kv_join, dim3((unsigned)(p.groups * chunks)), dim3(256), 0, st, a, wg_rows, p.nw / p.wr, chunks);
  return hipGetLastError();
}

}  // namespace qmv
