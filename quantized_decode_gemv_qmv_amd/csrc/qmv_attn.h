// qmv_attn.h -- host-side interface of the attention half of a decode layer
// (norm, cache append, attention) between the C ABI layer and its kernels.
// Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {

struct NormArgs {
  const float* x;
  int64_t ldx;
  const float* res;  // NULL, or fp32 [rows][ldr] added to x
  int64_t ldr;
  const float* w;  // [k]
  float eps;
  float* sum;  // NULL, or fp32 [rows][lds] that receives x + res
  int64_t lds;
  float* y;  // NULL, or fp32 [rows][ldy] that receives the normed rows
  int64_t ldy;
  int8_t* qs;
  float* d;
  int32_t* s;
  int rows, k;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st);

// The 8-bit cache and the sequences of one call (qmv_kv of the ABI).
struct KvView {
  int8_t* codes;         // [n_blocks][2][kvh][64 * dim]
  float* scales;         // [n_blocks][2][kvh]
  const int32_t* table;  // [n_seqs][width]
  const int32_t* lens;   // [n_seqs]
  const int32_t* start;  // NULL, or [n_seqs + 1]
  int64_t n_blocks;
  int kvh, dim, width, n_seqs, n_tok, max_q;
};

struct AppendArgs {
  KvView kv;
  const float* x[2];  // k and v
  int64_t ld[2];
};
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t st);

// Launch plan of the attention kernel: nw waves a workgroup, wr of them along
// the rows (16 each; the others along the cache blocks), row blocks of one
// (sequence, kv head), and the workgroups that share its cache blocks: splits
// for every group, or by length, as many as come to shares in all with parts
// of at least `least` blocks.
struct AttnPlan {
  int nw, wr, row_blocks, splits, shares, least;
  int64_t groups;    // n_seqs * kvh * row_blocks
  int64_t grid;      // workgroups with a workspace
  int64_t ws_bytes;  // 0: none is used
};
constexpr int64_t kAttnCounterBytes = 64 * 1024;
constexpr int kAttnMaxSplits = 64;  // one a lane where they are added up
AttnPlan attn_plan(int64_t n_seqs, int64_t max_q, int64_t n_heads, int64_t kvh, int64_t dim, int64_t width, int cus);

struct AttnArgs {
  KvView kv;
  const float* q;
  int64_t ldq;
  int group;        // query heads per kv head
  float scale;      // of the scores, times log2(e)
  int window;       // 0: none
  float* out;       // NULL, or fp32 [n_tok][ldo]
  int64_t ldo;
  int8_t* qs;       // NULL, or the Q8 blocks of the output rows
  float* qd;
  int32_t* qsum;
  int row_blocks, splits, shares, least;
  float* part;      // [workgroup][row][dim] unnormalized sums, then the
  float* ml;        // [workgroup][row][2] maxima and totals
  int* cnt;         // one arrival counter per group
};
hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t st);

}  // namespace qmv
