// qmv_steps.h -- host-side interface of the steps around a decode layer's
// matvecs (adapters, head norms with rotation, expert gates, log
// probabilities) between the C ABI layer and their kernels.  Not installed;
// not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {

// Norm and rotation of query and key heads.  Index 0: q, 1: k.
struct HeadsArgs {
  const float* x[2];  // [n_tok][ldx], head h at columns h * dim ..
  int64_t ldx[2];
  float* y[2];
  int64_t ldy[2];
  const float* w[2];  // NULL (no norm), or [dim]
  int heads[2];
  const int32_t* pos;   // NULL, or [n_axes][n_tok]
  const float* freq;    // [rot / 2]
  const int32_t* axis;  // NULL, or [rot / 2]
  int n_tok, dim, rot, n_axes;
  int adjacent;  // 1: pairs (2i, 2i + 1), 0: (i, i + rot / 2)
  float scale;   // of cos and sin
  double eps, inv_dim;
  int passes, waves_a_token;  // set at launch
};
hipError_t launch_head_norm_rope(const HeadsArgs& a, int cus, hipStream_t st);

// Low-rank adapters beside projections that share their input.
enum : int { kF16 = 0, kBF16 = 1, kF32 = 2 };  // qmv_float_type
constexpr int kLoraItems = 8;
struct LoraItem {
  const void* a;  // [adapters][max_rank][k]
  const void* b;  // [adapters][n][max_rank]
  const float* base;
  float* y;
  int64_t ldb, ldy;
  int n;
};
// What both kernels need.
struct LoraCall {
  const int32_t* ids;    // [n_tok]
  const int32_t* ranks;  // NULL, or [adapters]
  float* h;              // [slices][n_tok][n_items][max_rank]
  int32_t* tiles;        // [n_tok rounded up to 64][8]: a tile's tokens, adapter, rank, scale and the tokens
  int n_tok, n_items, adapters, max_rank;
  int slices, slots;  // of k, and of each 64 tokens; set at launch
};
struct LoraArgs {
  LoraCall call;
  LoraItem item[kLoraItems];
  const float* x;
  int64_t ldx;
  int k;
  const float* scales;  // NULL, or [adapters]
};
// The most partial sums of h that a call makes (k alone can make them fewer).
constexpr int kLoraMaxSlices = 16;
int lora_slices(int64_t n_items, int64_t max_rank, int64_t n_tok);
// Values of h that the workspace has room for.  Fewer rows take more slices, and
// can take more room: this one is that of any call of no more items, rank and rows.
int64_t lora_room(int64_t n_items, int64_t max_rank, int64_t n_tok);
hipError_t launch_lora(int type, LoraArgs& a, hipStream_t st);

// Routing to experts.
struct GateArgs {
  const float* x;  // [n_tok][ldx]
  int64_t ldx;
  const float* wr;  // [n_experts][k]
  int n_tok, k, n_experts, top_k;
  int sigmoid;         // 1: sigmoid scores, 0: softmax
  const float* bias;   // NULL, or [n_experts]
  int groups, top_groups, group_best;
  int renorm;
  float scale;
  int32_t* ids;       // [n_tok][top_k]
  float* weights;     // [n_tok][top_k]
  float* logits_out;  // NULL, or [n_tok][n_experts]
  int8_t* qs;         // NULL, or the Q8 blocks of x
  float* qd;
  int32_t* qsum;
  double* logits;  // [slices][n_tok][n_experts]
  int* cnt;        // the arrival counter
  int slices, slice;  // of k, and their length; set at launch
};
// The most slices of k that a call makes (k alone can make them fewer).
constexpr int kGateMaxSlices = 8;
int gate_slices(int64_t n_tok, int64_t n_experts);
// Logits that the workspace has room for: those of any call of no more tokens and experts.
int64_t gate_room(int64_t n_tok, int64_t n_experts);
hipError_t launch_router_gate(GateArgs a, hipStream_t st);

// Log probabilities of a row of logits.
constexpr int kPartGroupsOfRow = 32;  // keys of a part
struct LogprobArgs {
  const float* x;  // [n_tok][ldx]
  int64_t ldx;
  int n_tok, n_vocab;
  float scale;
  const int32_t* given;  // [n_tok][n_given]
  int n_given, top_n;
  float* logprobs;  // [n_tok][n_given]
  float* entropy;   // NULL, or [n_tok]
  int32_t* ids;     // [n_tok][top_n]
  float* top;       // [n_tok][top_n]
  int parts;        // of a row, 0: whole rows
  int loops;        // lengths of registers that a part has; set at launch
  float* sums;      // [n_tok][parts][4]
  uint64_t* keys;   // [n_tok][parts][kPartGroupsOfRow]
  int* cnt;         // arrival counters, kCounterStep apart
};
// Counters lie 256 bytes apart: the memory side takes the atomics of one line
// one after the other.
constexpr int kCounterStep = 64;
constexpr int kLogprobCounters = 256;  // rows in parts at most
// Parts of a row that a call with a workspace makes; 0: none.
int logprob_parts(int64_t n_tok, int64_t n_vocab, int64_t top_n);
// Parts that the workspace has room for: those of any call of no more rows and
// tokens; 0: none of them makes parts.
int64_t logprob_room(int64_t n_tok, int64_t n_vocab);
hipError_t launch_token_logprobs(LogprobArgs a, hipStream_t st);

}  // namespace qmv
