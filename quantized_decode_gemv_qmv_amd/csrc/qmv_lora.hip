// qmv_lora.hip -- low-rank adapters of many requests beside shared
// projections, for gfx950: y = base + scale * B (A x), each token with the A
// and B of its own adapter.
//
// Two launches: k_lora_down makes h = A x for all items and a list of the tiles
// that it found, k_lora_up the outputs.  A tile is up to four tokens that share
// an adapter among an aligned 64, so an adapter's weights are read once a tile, and
// tokens of different adapters cost no more than their own weights.  Weights enter
// as the fp32 numbers that they are and products and sums are fp32: nothing is
// rounded but sums.
//
// Bounds: two launches of some 2 us, each with a chain of loads (ids, ranks,
// weights; tile, h and weights) before it streams; for many adapters their bytes.
// 16 adapters of ranks up to 64 on 2 x 14336 rows (62 MB): 20.5 us, 3 TB/s; 64
// tokens of three adapters on 4096 x 14336: 11.6; 700 tokens: 23.
// Matrix instructions were measured and dropped: their operands want neighbouring
// lanes on different rows, which loads at a quarter of the rate (down, 700 tokens
// 10.4 -> 19 to 21 us), and through LDS the outputs of single tokens took longer
// (16 adapters 22.1 -> 24.2).
#include "qmv_device.h"
#include "qmv_steps.h"

namespace qmv {

namespace {

constexpr int kTile = 4;       // tokens of a tile
constexpr int kWaves = 4;      // of a workgroup
constexpr int kSlots = 24;     // workgroups that share 64 tokens: one each for the 16 to 23 tiles of up to eight adapters
constexpr int kCounted = 8;    // adapters of 64 tokens whose tokens are counted
constexpr int kDownRows = 4;   // of A in a wave
constexpr int kChunk = 512;    // columns of a wave's step: 8 a lane
constexpr int kUpThreads = 64 * kWaves;
constexpr int kUpAhead = 4;    // steps of rows whose loads are in flight
// Workgroups of a launch, about: more of them start more often, fewer leave
// compute units idle (outputs' target 256 / 512 / 1024 / 2048: 16 adapters 25 /
// 20.5 / 21.6 / 23.7 us, 700 tokens 26 / 23.0 / 23.7 / 24.9).
constexpr int64_t kDownTarget = 512, kUpTarget = 512;

// Kernel arguments.  The host writes them out at some 5 ns a byte, so a call's
// one to four items do not carry the room of eight (three items as one array of
// eight in both kernels: 10.7 us of host time a call, 6.0 as it is).
struct DownArgs {
  LoraCall c;
  const float* x;
  int64_t ldx;
  int k, slice;
  const float* scales;
  const void* a[kLoraItems];
};
struct UpItem {
  const void* b;
  const float* base;
  float* y;
  int64_t ldb, ldy;
  int n, first;  // first: of its workgroups along the outputs
};
template <int N>
struct UpArgs {
  LoraCall c;
  int steps;  // of rows that a workgroup takes
  UpItem item[N];
};

// Eight neighbouring weights as they lie in memory.
template <int DT>
struct Raw8 {
  u32x4 v[DT == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (DT == kF32) {
      v[0] = ld16(static_cast<const float*>(base) + at);
      v[1] = ld16(static_cast<const float*>(base) + at + 4);
    } else {
      v[0] = ld16(static_cast<const uint16_t*>(base) + at);
    }
  }
  __device__ __forceinline__ void clear() {
    v[0] = u32x4{0, 0, 0, 0};
    if constexpr (DT == kF32) v[1] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == kF32) return __uint_as_float(v[i / 4][i % 4]);
    if constexpr (DT == kF16) return half_bits_to_float(v[0][i / 2] >> (16 * (i & 1)));
    return __uint_as_float(i & 1 ? v[0][i / 2] & 0xFFFF0000u : v[0][i / 2] << 16);
  }
};

struct Tile {
  int n;        // tokens, 0: another workgroup has them
  int adapter;  // -1: none
  int rank;
  int tokens;   // lane j: the j-th one
  __device__ __forceinline__ int token(int j) const { return __builtin_amdgcn_readlane(tokens, min(j, n - 1)); }
};

// The aligned 64 tokens of a workgroup, one a lane.
struct Block {
  int base;
  int adapter;     // -1: none, -2: past the end
  int rank;
  bool start;      // whether the token may start a tile
  int place;       // among those
  uint64_t apart;  // tokens whose tiles are of neighbours only
  uint64_t turns;  // tokens whose adapter is not the one before's
};

// Tiles are of four tokens of an adapter wherever they stand among the 64 for
// the first kCounted adapters, whose tokens are counted; of neighbours for others,
// which takes no loop (a batch of many requests has each one's tokens side by
// side).  Where every token has a workgroup of its own each may start a tile, and
// tile_of looks whether it does.
__device__ __forceinline__ Block block_of(const LoraCall& a, int base) {
  const int lane = threadIdx.x & 63;
  Block b;
  b.base = base;
  b.adapter = -2;
  if (base + lane < a.n_tok) {
    const int id = a.ids[base + lane];
    b.adapter = id < 0 || id >= a.adapters ? -1 : id;
  }
  b.rank = 0;
  if (b.adapter >= 0) b.rank = a.ranks != nullptr ? max(0, min(a.ranks[b.adapter], a.max_rank)) : a.max_rank;
  const uint64_t below = (1ull << lane) - 1;
  uint64_t left = __ballot(b.adapter != -2), starts = left;
  b.apart = b.turns = 0;
  if (a.n_tok > a.slots) {  // uniform
    starts = 0;
    for (int i = 0; i < kCounted && left != 0; ++i) {
      const int id = __builtin_amdgcn_readlane(b.adapter, __ffsll((unsigned long long)left) - 1);
      const uint64_t m = __ballot(b.adapter == id);
      starts |= __ballot(b.adapter == id && __popcll(m & below) % kTile == 0);
      left &= ~m;
    }
    if (left != 0) {
      const int before = __shfl_up(b.adapter, 1, 64);
      b.turns = __ballot(lane == 0 || before != b.adapter);
      const int first = 63 - __clzll((long long)(b.turns & (below | 1ull << lane)));
      b.apart = left;
      starts |= __ballot((lane - first) % kTile == 0) & left;
    }
  }
  b.start = (starts >> lane) & 1;
  b.place = (int)__popcll(starts & below);
  return b;
}

// The block's tile at place `place`; false: there is none any more.
__device__ __forceinline__ bool tile_of(const Block& b, int place, Tile& r) {
  const int lane = threadIdx.x & 63;
  const uint64_t here = __ballot(b.start && b.place == place);
  if (here == 0) return false;
  const int at = __ffsll((unsigned long long)here) - 1;
  r.adapter = __builtin_amdgcn_readlane(b.adapter, at);
  r.rank = __builtin_amdgcn_readlane(b.rank, at);
  if ((b.apart >> at) & 1) {  // neighbours, up to where the adapter changes
    const uint64_t next = at < 63 ? b.turns >> (at + 1) : 0;
    r.n = min(next != 0 ? __ffsll((unsigned long long)next) : 64 - at, kTile);
    r.tokens = b.base + at + lane;
    return true;
  }
  uint64_t m = __ballot(b.adapter == r.adapter);
  const int before = (int)__popcll(m & ((1ull << at) - 1));
  m &= ~0ull << at;
  r.n = before % kTile == 0 ? min((int)__popcll(m), kTile) : 0;
  // each of them writes its number to the lane of its place; the others go to
  // the last lane, which is a place only if there are no others
  const int to = (m >> lane) & 1 ? (int)__popcll(m & ((1ull << lane) - 1)) : 63;
  r.tokens = __builtin_amdgcn_ds_permute(4 * to, b.base + lane);
  return true;
}

// TG tokens by kDownRows rows of A over the columns lo .. hi - 1: the sums in
// lane row * TG + token.  All loads of a step are in flight together.
template <int DT, int TG>
__device__ __forceinline__ float down(const DownArgs& a, const void* w, const int64_t (&row)[kDownRows],
                                      const Tile& tile, int lo, int hi) {
  constexpr int U = TG == 1 ? 2 : 1;  // steps whose loads are in flight
  const int lane = threadIdx.x & 63;
  float acc[kDownRows * TG];
#pragma unroll
  for (int i = 0; i < kDownRows * TG; ++i) acc[i] = 0.f;
  int64_t col[TG];
#pragma unroll
  for (int j = 0; j < TG; ++j) col[j] = tile.token(j) * a.ldx;
  for (int c0 = lo + 8 * lane; c0 < hi; c0 += U * kChunk) {
    Raw8<DT> wv[U][kDownRows];
    Raw8<kF32> xv[U][TG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kChunk;
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) wv[u][r].clear();
#pragma unroll
      for (int j = 0; j < TG; ++j) xv[u][j].clear();
      if (u == 0 || c < hi) {
#pragma unroll
        for (int r = 0; r < kDownRows; ++r) wv[u][r].load(w, row[r] + c);
#pragma unroll
        for (int j = 0; j < TG; ++j) xv[u][j].load(a.x, col[j] + c);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < kDownRows; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wf = wv[u][r].get(i);
#pragma unroll
          for (int j = 0; j < TG; ++j) acc[r * TG + j] = fmaf(wf, xv[u][j].get(i), acc[r * TG + j]);
        }
  }
  return fold_all<kDownRows * TG>(acc, lane);
}

}  // namespace

// h[slice][t][item][r] = sum over the slice's columns of A[r][c] x[t][c]: a
// wave for four rows, the workgroup's waves side by side over the same columns,
// so that x comes from memory once for 16 rows.
template <int DT>
__global__ __launch_bounds__(64 * kWaves) void k_lora_down(DownArgs a) {
  const int groups = (a.c.max_rank + kDownRows * kWaves - 1) / (kDownRows * kWaves);
  const int item = blockIdx.x / groups;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r0 = (blockIdx.x % groups) * kDownRows * kWaves + __builtin_amdgcn_readfirstlane(wave) * kDownRows;
  const int lo = blockIdx.z * a.slice, hi = min(lo + a.slice, a.k);
  const Block block = block_of(a.c, (int)blockIdx.y / a.c.slots * 64);
  const void* w = a.a[item];
  Tile tile;
  int p = (int)blockIdx.y % a.c.slots;
  for (; tile_of(block, p, tile); p += a.c.slots) {
    const int n = tile.n, rank = tile.rank;
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x < 8) {
      const int f = threadIdx.x;
      const int token = __shfl(tile.tokens, max(0, min(f - 4, n - 1)));  // with every lane that holds one on
      const int scale = tile.adapter >= 0 && a.scales != nullptr ? __float_as_int(a.scales[tile.adapter]) : 0x3F800000;
      const int v = f == 0 ? n : f == 1 ? tile.adapter : f == 2 ? rank : f == 3 ? scale : token;
      a.c.tiles[8 * (block.base + p) + f] = v;
    }
    if (n == 0 || r0 >= rank) continue;
    int64_t row[kDownRows];
#pragma unroll
    for (int r = 0; r < kDownRows; ++r)  // rows past the rank repeat the last one
      row[r] = ((int64_t)tile.adapter * a.c.max_rank + min(r0 + r, rank - 1)) * a.k;
    float s;
    int tg;
    if (n == 1) {
      tg = 1;
      s = down<DT, 1>(a, w, row, tile, lo, hi);
    } else if (n == 2) {
      tg = 2;
      s = down<DT, 2>(a, w, row, tile, lo, hi);
    } else {
      tg = 4;
      s = down<DT, 4>(a, w, row, tile, lo, hi);
    }
    const int r = r0 + lane / tg, j = lane % tg;
    const int at = __shfl(tile.tokens, j);
    if (lane < kDownRows * tg && r < rank && j < n)
      a.c.h[(((int64_t)blockIdx.z * a.c.n_tok + at) * a.c.n_items + item) * a.c.max_rank + r] = s;
  }
  // the end of the slot's list
  if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0 && p < 64) a.c.tiles[8 * (block.base + p)] = -1;
}

namespace {

// The partner whose bit H differs: a mirror where no exchange of that distance
// exists (every lane below that bit holds the same kind of value).
template <int H>
__device__ __forceinline__ float partner(float v) {
  if constexpr (H == 1) return dpp_f<DPP_XOR1>(v);
  if constexpr (H == 2) return dpp_f<DPP_XOR2>(v);
  if constexpr (H == 4) return dpp_f<DPP_HALF_MIRROR>(v);
  if constexpr (H == 8) return dpp_f<DPP_MIRROR>(v);
  return __shfl_xor(v, H, 64);
}

// Sums of N values over a lane group of 2 H lanes.  While a lane has several
// values, it keeps one half of them and gives the other away; `at` counts up
// the place of the first one that it keeps, `own` whether it is to store them.
template <int H, int N>
__device__ __forceinline__ void fold_group(float* v, int lane, int& at, bool& own) {
  if constexpr (H >= 1) {
    const bool hi = (lane & H) != 0;
    if constexpr (N > 1) {
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float send = hi ? v[j] : v[j + N / 2];
        const float keep = hi ? v[j + N / 2] : v[j];
        v[j] = keep + partner<H>(send);
      }
      at += hi ? N / 2 : 0;
      fold_group<H / 2, N / 2>(v, lane, at, own);
    } else {
      v[0] += partner<H>(v[0]);
      own = own && !hi;
      fold_group<H / 2, 1>(v, lane, at, own);
    }
  }
}

// The outputs of a tile of at most TG tokens: steps of kUpThreads / LPR rows, LPR
// lanes a row, TG tokens at once.  The weights and base of kUpAhead steps are
// on their way while one is worked on.
template <int DT, int LPR, int TG>
__device__ __forceinline__ void up(const LoraCall& a, float scale, const UpItem& it, int m, const Tile& tile, int rank, float* hs,
                                   int n0, int steps) {
  constexpr int OWN = TG > LPR ? TG / LPR : 1;  // values that a lane stores
  constexpr int kStep = kUpThreads / LPR;
  const int l = threadIdx.x % LPR, row = n0 + (int)threadIdx.x / LPR;
  int at = 0;
  bool own = true;
  {
    float none[TG] = {};
    fold_group<LPR / 2, TG>(none, l, at, own);
  }
  const char* wp = static_cast<const char*>(it.b) + (int64_t)tile.adapter * it.n * a.max_rank * (DT == kF32 ? 4 : 2);
  const float* bp[OWN];
  float* yp[OWN];
  bool ok[OWN];
#pragma unroll
  for (int j = 0; j < OWN; ++j) {
    const int t = __shfl(tile.tokens, min(at + j, tile.n - 1));
    bp[j] = it.base + t * it.ldb;
    yp[j] = it.y + t * it.ldy;
    ok[j] = own && at + j < tile.n;
  }
  Raw8<DT> b[kUpAhead];
  float base[kUpAhead][OWN];
  auto fetch = [&](int s, Raw8<DT>& w, float (&v)[OWN]) {
    const int r = row + s * kStep;
    w.clear();
#pragma unroll
    for (int j = 0; j < OWN; ++j) v[j] = 0.f;
    if (s < steps && r < it.n) {
      if (8 * l < rank) w.load(wp, (int64_t)r * a.max_rank + 8 * l);
      if (it.base != nullptr) {
#pragma unroll
        for (int j = 0; j < OWN; ++j)
          if (ok[j]) v[j] = bp[j][r];
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kUpAhead; ++i) fetch(i, b[i], base[i]);
  __syncthreads();  // the tile before is done with hs
  // h: the slices' sums, eight loads in flight
  const int64_t step = (int64_t)a.n_tok * a.n_items * a.max_rank;
  for (int e = threadIdx.x; e < TG * 8 * LPR; e += kUpThreads) {
    const int j = e / (8 * LPR), r = e % (8 * LPR);
    float v = 0.f;
    const int t = __shfl(tile.tokens, min(j, tile.n - 1));
    if (r < rank && j < tile.n) {
      const float* p = a.h + ((int64_t)t * a.n_items + m) * a.max_rank + r;
      for (int z0 = 0; z0 < a.slices; z0 += 8) {
        float u[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) u[z] = p[min(z0 + z, a.slices - 1) * step];
#pragma unroll
        for (int z = 0; z < 8; ++z) v += z0 + z < a.slices ? u[z] : 0.f;
      }
    }
    hs[e] = v;
  }
  __syncthreads();
  float h[TG][8];
#pragma unroll
  for (int j = 0; j < TG; ++j) {
    const f32x4* p = reinterpret_cast<const f32x4*>(hs + j * 8 * LPR + 8 * l);
    const f32x4 u = p[0], v = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[j][i] = u[i];
      h[j][4 + i] = v[i];
    }
  }
  for (int s0 = 0; s0 < steps; s0 += kUpAhead) {
#pragma unroll
    for (int i = 0; i < kUpAhead; ++i) {
      if (s0 + i < steps) {  // uniform
        const int r = row + (s0 + i) * kStep;
        float s[TG];
#pragma unroll
        for (int j = 0; j < TG; ++j) s[j] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = 8 * l + e < rank ? b[i].get(e) : 0.f;  // columns past the rank may hold anything
#pragma unroll
          for (int j = 0; j < TG; ++j) s[j] = fmaf(w, h[j][e], s[j]);
        }
        int unused = 0;
        bool skip = true;
        fold_group<LPR / 2, TG>(s, l, unused, skip);
        float y[OWN];
#pragma unroll
        for (int j = 0; j < OWN; ++j) y[j] = fmaf(scale, s[j], base[i][j]);
        fetch(s0 + i + kUpAhead, b[i], base[i]);
#pragma unroll
        for (int j = 0; j < OWN; ++j)
          if (ok[j] && r < it.n) yp[j][r] = y[j];
      }
    }
  }
}

}  // namespace

// y[t][r] = base[t][r] + scale * sum over i of B[r][i] h[t][i]: a workgroup
// takes `steps` steps of an item's rows for a tile.
template <int DT, int LPR, int N>
__global__ __launch_bounds__(kUpThreads) void k_lora_up(UpArgs<N> a) {
  __shared__ __align__(16) float hs[kTile * 8 * LPR];
  int m = 0;
#pragma unroll
  for (int i = 1; i < N; ++i) m += i < a.c.n_items && (int)blockIdx.x >= a.item[i].first ? 1 : 0;
  const UpItem it = a.item[m];
  const int n0 = ((int)blockIdx.x - it.first) * (kUpThreads / LPR) * a.steps;
  const int rows = min(kUpThreads / LPR * a.steps, it.n - n0);
  const int base = (int)blockIdx.y / a.c.slots * 64;
  for (int p = (int)blockIdx.y % a.c.slots; p < 64; p += a.c.slots) {
    // the list that k_lora_down wrote, through the scalar cache
    typedef const __attribute__((address_space(4))) int* Scalars;
    const Scalars f = (Scalars)(uintptr_t)(a.c.tiles + 8 * (base + p));
    Tile tile;
    tile.n = f[0];
    tile.adapter = f[1];
    tile.rank = f[2];
    const float scale = __int_as_float(f[3]);
    const int lane = threadIdx.x & 3;
    const int t0 = f[4], t1 = f[5], t2 = f[6], t3 = f[7];
    tile.tokens = lane < 2 ? (lane == 0 ? t0 : t1) : (lane == 2 ? t2 : t3);
    if (tile.n < 0) break;
    if (tile.n == 0) continue;
    const int rank = tile.rank;
    if (rank == 0) {  // no adapter: y = base
      if (it.y == it.base) continue;
      for (int j = 0; j < tile.n; ++j) {
        const int s = tile.token(j);
        for (int r = n0 + threadIdx.x; r < n0 + rows; r += kUpThreads)
          it.y[s * it.ldy + r] = it.base != nullptr ? it.base[s * it.ldb + r] : 0.f;
      }
      continue;
    }
    const int steps = (rows + kUpThreads / LPR - 1) / (kUpThreads / LPR);
    if (tile.n == 1) up<DT, LPR, 1>(a.c, scale, it, m, tile, rank, hs, n0, steps);
    else if (tile.n == 2) up<DT, LPR, 2>(a.c, scale, it, m, tile, rank, hs, n0, steps);
    else up<DT, LPR, 4>(a.c, scale, it, m, tile, rank, hs, n0, steps);
  }
}

// Tiles that a call's tokens are taken to make: one of n_tok / kTile .. n_tok,
// which the ids decide.
static int64_t likely_tiles(int64_t n_tok) {
  const int64_t few = n_tok < 8 ? n_tok : 8, least = (n_tok + kTile - 1) / kTile;
  return few > least ? few : least;
}

int lora_slices(int64_t n_items, int64_t max_rank, int64_t n_tok) {
  const int64_t rows = kDownRows * kWaves;
  const int64_t groups = n_items * ((max_rank + rows - 1) / rows) * likely_tiles(n_tok);
  const int64_t want = (kDownTarget + groups - 1) / groups;
  return (int)(want > kLoraMaxSlices ? kLoraMaxSlices : want);
}

// With g groups, rank <= 16 g / (items * tiles) and g * slices is below g +
// kDownTarget and 16 g at most; rows / tiles is 1 up to 8 rows, rows / 8 up to 32
// and at most 4 from there on.  None of it falls as an argument grows.
int64_t lora_room(int64_t n_items, int64_t max_rank, int64_t n_tok) {
  const int64_t rows = kDownRows * kWaves;
  const int64_t g = n_items * ((max_rank + rows - 1) / rows) * likely_tiles(n_tok);
  const int64_t most = g * kLoraMaxSlices, near = g + kDownTarget - 1;
  const int64_t eighths = n_tok < 8 ? 8 : (n_tok < kTile * 8 ? n_tok : kTile * 8);
  return rows * (most < near ? most : near) * eighths / 8;
}

namespace {

template <int DT, int LPR, int N>
hipError_t launch_up(const LoraArgs& a, hipStream_t st) {
  constexpr int kStep = kUpThreads / LPR;
  UpArgs<N> u{};
  u.c = a.call;
  int64_t steps = 0;
  for (int i = 0; i < a.call.n_items; ++i) steps += (a.item[i].n + kStep - 1) / kStep;
  const int64_t tiles = likely_tiles(a.call.n_tok), want = (kUpTarget + tiles - 1) / tiles;
  u.steps = (int)((steps + want - 1) / want);
  int64_t wgs = 0;
  for (int i = 0; i < a.call.n_items; ++i) {
    const LoraItem& m = a.item[i];
    u.item[i] = UpItem{m.b, m.base, m.y, m.ldb, m.ldy, m.n, (int)wgs};
    wgs += (m.n + kStep * u.steps - 1) / (kStep * u.steps);
  }
  hipLaunchKernelGGL((k_lora_up<DT, LPR, N>), dim3((unsigned)wgs, (unsigned)((a.call.n_tok + 63) / 64 * a.call.slots)), dim3(kUpThreads), 0, st, u);
  return hipGetLastError();
}

template <int DT, int N>
hipError_t launch_up(const LoraArgs& a, hipStream_t st) {
  const int v = a.call.max_rank / 8;
  if (v <= 1) return launch_up<DT, 1, N>(a, st);
  if (v <= 2) return launch_up<DT, 2, N>(a, st);
  if (v <= 4) return launch_up<DT, 4, N>(a, st);
  if (v <= 8) return launch_up<DT, 8, N>(a, st);
  if (v <= 16) return launch_up<DT, 16, N>(a, st);
  return launch_up<DT, 32, N>(a, st);
}

template <int DT>
hipError_t launch(LoraArgs& a, hipStream_t st) {
  DownArgs d{};
  // slices of whole chunks
  const int most = (a.k + kChunk - 1) / kChunk;
  const int want = min(lora_slices(a.call.n_items, a.call.max_rank, a.call.n_tok), most);
  d.slice = (most + want - 1) / want * kChunk;
  a.call.slices = (a.k + d.slice - 1) / d.slice;
  a.call.slots = min(a.call.n_tok, kSlots);
  d.c = a.call;
  d.x = a.x;
  d.ldx = a.ldx;
  d.k = a.k;
  d.scales = a.scales;
  for (int i = 0; i < a.call.n_items; ++i) d.a[i] = a.item[i].a;
  const int rows = kDownRows * kWaves, groups = (a.call.max_rank + rows - 1) / rows;
  hipLaunchKernelGGL((k_lora_down<DT>),
                     dim3((unsigned)(a.call.n_items * groups), (unsigned)((a.call.n_tok + 63) / 64 * a.call.slots), (unsigned)a.call.slices),
                     dim3(64 * kWaves), 0, st, d);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return a.call.n_items <= 4 ? launch_up<DT, 4>(a, st) : launch_up<DT, kLoraItems>(a, st);
}

}  // namespace

hipError_t launch_lora(int type, LoraArgs& a, hipStream_t st) {
  if (type == kF16) return launch<kF16>(a, st);
  if (type == kBF16) return launch<kBF16>(a, st);
  return launch<kF32>(a, st);
}

}  // namespace qmv
