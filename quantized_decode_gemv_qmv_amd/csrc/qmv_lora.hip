// qmv_lora.hip -- low-rank adapters of many requests beside shared
// projections, for gfx950: y = base + scale * B (A x), each token with the A
// and B of its own adapter.
//
// Two launches: k_lora_down makes h = A x for all items, k_lora_up the outputs.
// Both work on tiles of up to kTile tokens that share an adapter, found from
// the ids of their aligned 64 tokens: a workgroup belongs to a token, and goes
// on if as many tokens before it as a whole number of tiles hold its adapter.
// So an adapter's weights are read once a tile, and tokens of different
// adapters cost no more than their own weights.
#include "qmv_device.h"
#include "qmv_steps.h"

namespace qmv {

namespace {

constexpr int kTile = 8;      // tokens of a tile
constexpr int kDownWaves = 4;
constexpr int kDownRows = 4;  // of A in a workgroup
constexpr int kChunk = 512;   // columns of a wave's step: 8 a lane
constexpr int kUpThreads = 256;

// Eight neighbouring weights as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&o)[8]) {
  if constexpr (DT == kF32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
    const f32x4 u = p[0], v = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = u[i];
      o[4 + i] = v[i];
    }
  } else {
    const u32x4 u = ld16(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kF16) {
        o[2 * i] = half_bits_to_float(u[i]);
        o[2 * i + 1] = half_bits_to_float(u[i] >> 16);
      } else {
        o[2 * i] = __uint_as_float(u[i] << 16);
        o[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
  }
}

struct Tile {
  int n;         // tokens, 0: another workgroup has them
  int adapter;   // -1: none
  uint64_t left; // of the 64 tokens, this tile's
  int base;      // the first of the 64
};

// The tile of token t, in every wave alike.
__device__ __forceinline__ Tile tile_of(const LoraArgs& a, int t) {
  const int lane = threadIdx.x & 63, base = t & ~63;
  int id = -2;
  if (base + lane < a.n_tok) {
    id = a.ids[base + lane];
    if (id < 0 || id >= a.adapters) id = -1;
  }
  const int mine = __builtin_amdgcn_readlane(id, t & 63);
  uint64_t m = __ballot(id == mine);
  const int before = __popcll(m & ((1ull << (t & 63)) - 1));
  Tile r{0, mine, 0, base};
  if (before % kTile != 0) return r;
  m &= ~0ull << (t & 63);
  r.n = min(__popcll(m), kTile);
  r.left = m;
  return r;
}

__device__ __forceinline__ int next_token(Tile& t) {
  const int i = __ffsll((unsigned long long)t.left) - 1;
  t.left &= t.left - 1;
  return t.base + i;
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
  if (adapter < 0) return 0;
  if (a.ranks == nullptr) return a.max_rank;
  return max(0, min(a.ranks[adapter], a.max_rank));
}

// TG tokens (the first n count) by kDownRows rows of A over this wave's part
// of a slice: the sums in lane row * TG + token.
template <int DT, int TG>
__device__ __forceinline__ float down(const LoraArgs& a, const void* w, const int64_t (&row)[kDownRows],
                                      const int (&tok)[kTile], int lo, int hi) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float acc[kDownRows * TG];
#pragma unroll
  for (int i = 0; i < kDownRows * TG; ++i) acc[i] = 0.f;
  for (int c = lo + kChunk * wave + 8 * lane; c < hi; c += kChunk * kDownWaves) {
    float wv[kDownRows][8];
#pragma unroll
    for (int r = 0; r < kDownRows; ++r) load8<DT>(w, row[r] + c, wv[r]);
#pragma unroll
    for (int j = 0; j < TG; ++j) {
      float xv[8];
      load8<kF32>(a.x, tok[j] * a.ldx + c, xv);
#pragma unroll
      for (int r = 0; r < kDownRows; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r * TG + j] = fmaf(wv[r][i], xv[i], acc[r * TG + j]);
    }
  }
  return fold_all<kDownRows * TG>(acc, lane);
}

}  // namespace

// h[slice][t][item][r] = sum over the slice's columns of A[r][c] x[t][c]:
// workgroups along (item, rows), tokens and slices; four waves share a slice.
template <int DT>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraArgs a) {
  __shared__ float part[kDownWaves][kDownRows * kTile];
  Tile tile = tile_of(a, blockIdx.y);
  const int groups = (a.max_rank + kDownRows - 1) / kDownRows;
  const int item = blockIdx.x / groups, r0 = (blockIdx.x % groups) * kDownRows;
  const int rank = rank_of(a, tile.adapter);
  if (tile.n == 0 || r0 >= rank) return;
  int64_t row[kDownRows];
#pragma unroll
  for (int r = 0; r < kDownRows; ++r)  // rows past the rank repeat the last one
    row[r] = ((int64_t)tile.adapter * a.max_rank + min(r0 + r, rank - 1)) * a.k;
  int tok[kTile];
#pragma unroll
  for (int j = 0; j < kTile; ++j) tok[j] = j < tile.n ? next_token(tile) : tok[0];
  const int lo = blockIdx.z * a.slice, hi = min(lo + a.slice, a.k);
  const void* w = a.item[item].a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float s;
  int tg;
  if (tile.n == 1) {
    tg = 1;
    s = down<DT, 1>(a, w, row, tok, lo, hi);
  } else if (tile.n == 2) {
    tg = 2;
    s = down<DT, 2>(a, w, row, tok, lo, hi);
  } else if (tile.n <= 4) {
    tg = 4;
    s = down<DT, 4>(a, w, row, tok, lo, hi);
  } else {
    tg = 8;
    s = down<DT, 8>(a, w, row, tok, lo, hi);
  }
  if (lane < kDownRows * tg) part[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x < kDownRows * tg) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kDownWaves; ++i) v += part[i][threadIdx.x];
    const int r = r0 + threadIdx.x / tg, j = threadIdx.x % tg;
    int t = tok[0];
#pragma unroll
    for (int i = 1; i < kTile; ++i) t = i == j ? tok[i] : t;
    if (r < rank && j < tile.n)
      a.h[(((int64_t)blockIdx.z * a.n_tok + t) * a.n_items + item) * a.max_rank + r] = v;
  }
}

namespace {

template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LPR >= 2) v += dpp_f<DPP_XOR1>(v);
  if constexpr (LPR >= 4) v += dpp_f<DPP_XOR2>(v);
  if constexpr (LPR >= 8) v += dpp_f<DPP_HALF_MIRROR>(v);
  if constexpr (LPR >= 16) v += dpp_f<DPP_MIRROR>(v);
  if constexpr (LPR >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// RPT rows a lane group, LPR lanes a row, TG tokens (the first n count).
template <int DT, int LPR, int RPT, int TG>
__device__ __forceinline__ void up(const LoraArgs& a, const LoraItem& it, const float* hs, int adapter, int rank,
                                   int n, const int (&tok)[kTile], int n0) {
  const int l = threadIdx.x % LPR, c = 8 * l;
  const float scale = a.scales != nullptr ? a.scales[adapter] : 1.f;
  float h[TG][8];
#pragma unroll
  for (int j = 0; j < TG; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = hs[j * 8 * LPR + c + i];
  float b[RPT][8];
#pragma unroll
  for (int q = 0; q < RPT; ++q) {
    const int r = min(n0 + q * (kUpThreads / LPR) + (int)threadIdx.x / LPR, it.n - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[q][i] = 0.f;
    if (c < rank) load8<DT>(it.b, ((int64_t)adapter * it.n + r) * a.max_rank + c, b[q]);
    // columns past the rank may hold anything
#pragma unroll
    for (int i = 0; i < 8; ++i) b[q][i] = c + i < rank ? b[q][i] : 0.f;
  }
#pragma unroll
  for (int q = 0; q < RPT; ++q) {
    const int r = n0 + q * (kUpThreads / LPR) + (int)threadIdx.x / LPR;
    const bool ok = r < it.n;
    float base[TG], s[TG];
#pragma unroll
    for (int j = 0; j < TG; ++j) {
      base[j] = 0.f;
      if (ok && j < n && j % LPR == l && it.base != nullptr) base[j] = it.base[tok[j] * it.ldb + r];
    }
#pragma unroll
    for (int j = 0; j < TG; ++j) {
      s[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j] = fmaf(b[q][i], h[j][i], s[j]);
      s[j] = lanes_sum<LPR>(s[j]);
    }
#pragma unroll
    for (int j = 0; j < TG; ++j)
      if (ok && j < n && j % LPR == l) it.y[tok[j] * it.ldy + r] = fmaf(scale, s[j], base[j]);
  }
}

}  // namespace

// y[t][r] = base[t][r] + scale * sum over i of B[r][i] h[t][i].
template <int DT, int LPR, int RPT>
__global__ __launch_bounds__(kUpThreads) void k_lora_up(LoraArgs a) {
  __shared__ float hs[kTile * 8 * LPR];
  Tile tile = tile_of(a, blockIdx.y);
  if (tile.n == 0) return;
  int m = 0;
  for (int i = 1; i < a.n_items; ++i) m += (int)blockIdx.x >= a.item[i].first ? 1 : 0;
  const LoraItem it = a.item[m];
  const int rank = rank_of(a, tile.adapter), n = tile.n;
  const int n0 = ((int)blockIdx.x - it.first) * (kUpThreads / LPR) * RPT;
  int tok[kTile];
#pragma unroll
  for (int j = 0; j < kTile; ++j) tok[j] = j < n ? next_token(tile) : tok[0];
  if (rank == 0) {  // no adapter: y = base
    if (it.y == it.base) return;
    for (int j = 0; j < n; ++j) {
      const int t = tok[0];
#pragma unroll
      for (int i = 0; i + 1 < kTile; ++i) tok[i] = tok[i + 1];
      for (int r = n0 + threadIdx.x; r < min(n0 + kUpThreads / LPR * RPT, it.n); r += kUpThreads)
        it.y[t * it.ldy + r] = it.base != nullptr ? it.base[t * it.ldb + r] : 0.f;
    }
    return;
  }
  for (int i = threadIdx.x; i < kTile * 8 * LPR; i += kUpThreads) {
    const int j = i / (8 * LPR), r = i % (8 * LPR);
    float v = 0.f;
    if (j < n && r < rank) {
      int t = tok[0];
#pragma unroll
      for (int q = 1; q < kTile; ++q) t = q == j ? tok[q] : t;
      const int64_t step = (int64_t)a.n_tok * a.n_items * a.max_rank;
      const float* p = a.h + ((int64_t)t * a.n_items + m) * a.max_rank + r;
      for (int z = 0; z < a.slices; ++z) v += p[z * step];
    }
    hs[i] = v;
  }
  __syncthreads();
  if (n == 1) up<DT, LPR, RPT, 1>(a, it, hs, tile.adapter, rank, n, tok, n0);
  else if (n == 2) up<DT, LPR, RPT, 2>(a, it, hs, tile.adapter, rank, n, tok, n0);
  else if (n <= 4) up<DT, LPR, RPT, 4>(a, it, hs, tile.adapter, rank, n, tok, n0);
  else up<DT, LPR, RPT, 8>(a, it, hs, tile.adapter, rank, n, tok, n0);
}

int lora_slices(int64_t n_items, int64_t max_rank, int64_t n_tok) {
  // about two workgroups a compute unit at the fewest tiles that the tokens can make
  const int64_t groups = n_items * ((max_rank + kDownRows - 1) / kDownRows) * ((n_tok + kTile - 1) / kTile);
  const int64_t want = (512 + groups - 1) / groups;
  return (int)(want > kLoraMaxSlices ? kLoraMaxSlices : want);
}

namespace {

template <int DT, int LPR, int RPT>
hipError_t launch_up(LoraArgs& a, hipStream_t st) {
  const int rows = kUpThreads / LPR * RPT;
  int64_t wgs = 0;
  for (int i = 0; i < a.n_items; ++i) {
    a.item[i].first = (int)wgs;
    wgs += (a.item[i].n + rows - 1) / rows;
  }
  hipLaunchKernelGGL((k_lora_up<DT, LPR, RPT>), dim3((unsigned)wgs, (unsigned)a.n_tok), dim3(kUpThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT, int LPR>
hipError_t launch_up(LoraArgs& a, hipStream_t st) {
  int64_t rows = 0;
  for (int i = 0; i < a.n_items; ++i) rows += a.item[i].n;
  // four rows a lane group once that leaves four workgroups a compute unit
  if (rows * LPR / kUpThreads / 4 * ((a.n_tok + kTile - 1) / kTile) >= 1024) return launch_up<DT, LPR, 4>(a, st);
  return launch_up<DT, LPR, 1>(a, st);
}

template <int DT>
hipError_t launch(LoraArgs a, hipStream_t st) {
  const int groups = (a.max_rank + kDownRows - 1) / kDownRows;
  hipLaunchKernelGGL((k_lora_down<DT>), dim3((unsigned)(a.n_items * groups), (unsigned)a.n_tok, (unsigned)a.slices),
                     dim3(64 * kDownWaves), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int v = a.max_rank / 8;
  if (v <= 1) return launch_up<DT, 1>(a, st);
  if (v <= 2) return launch_up<DT, 2>(a, st);
  if (v <= 4) return launch_up<DT, 4>(a, st);
  if (v <= 8) return launch_up<DT, 8>(a, st);
  if (v <= 16) return launch_up<DT, 16>(a, st);
  return launch_up<DT, 32>(a, st);
}

}  // namespace

hipError_t launch_lora(int type, LoraArgs a, hipStream_t st) {
  // as many slices as have a chunk for every wave
  const int most = (a.k + kChunk * kDownWaves - 1) / (kChunk * kDownWaves);
  a.slices = min(lora_slices(a.n_items, a.max_rank, a.n_tok), most);
  a.slice = ((a.k + a.slices - 1) / a.slices + kChunk - 1) / kChunk * kChunk;
  if (type == kF16) return launch<kF16>(a, st);
  if (type == kBF16) return launch<kBF16>(a, st);
  return launch<kF32>(a, st);
}

}  // namespace qmv
