// Internal launch interface of the experts' layers and the balance loss
// (ep_mi355x_expert.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ep_layer.h"

namespace ep {

// EP_ACT_*
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

// One of the three products of an expert's layer.  Forward: rows are x's,
// columns the output's.  grad_x: rows are grad_pre's, columns x's, the
// contraction runs over the W outputs.  grad_w: rows are the W outputs,
// columns x's, the contraction runs over the expert's rows.
struct LinearArgs {
  const uint16_t* x;  // bf16 rows, row stride ldx
  int64_t ldx;
  const int32_t* xmap;  // row of x for each expert-major row; null: itself
  const uint16_t* g;    // backward: bf16 grad_pre rows, row stride ldg
  int64_t ldg;
  const uint16_t* w;     // bf16 [E, W, H]
  const uint16_t* bias;  // bf16 [E, W] or null
  const uint16_t* res;   // bf16 rows of N, row stride ldres, or null
  int64_t ldres;
  uint16_t* out;  // forward: rows of N; grad_x: rows of H; row stride ldout
  int64_t ldout;
  uint16_t* pre;  // rows of W, row stride ldpre, or null
  int64_t ldpre;
  uint16_t* gw;  // grad_w [E, W, H]
  uint16_t* gb;  // grad_bias [E, W] or null
  float* part;   // grad_w: workspace, fp32 partial sums [splits][E][W][H], then [splits][E][W] of the bias
  int splits;    // parts of each expert's rows (grad_w)
  int run;       // tiles that an XCD takes in a row
  int32_t* even;  // grad_w: 0 there: runs of 32 instead; null: as run says
  const int32_t* counts;
  const int32_t* offsets;
  int E, H, N, W;  // W: N, or 2 N if gated
  int act;
  bool gated;
  int32_t* status;
  uint32_t generation;
};

// grad_pre = grad_out times the activation's derivative, over the rows of a
// selection.
struct ActBackwardArgs {
  const uint16_t* go;
  int64_t ldgo;
  const uint16_t* pre;
  int64_t ldpre;
  uint16_t* gpre;
  int64_t ldgpre;
  const int32_t* counts;
  const int32_t* offsets;
  int E, N, act;
  bool gated;
  bool padded;  // segments are aligned: rows of no selection lie between them
  int32_t* status;
  uint32_t generation;
};

// rows: of a selection, at most
hipError_t launch_linear(const LinearArgs& a, int64_t rows, hipStream_t s);
// grad_x of x and grad_w of w, either null
hipError_t launch_linear_grads(const LinearArgs* x, const LinearArgs* w, int64_t rows, hipStream_t s);
// rows: up to offsets[E], at most
hipError_t launch_act_backward(const ActBackwardArgs& a, int64_t rows, hipStream_t s);

// The balance loss.  Tokens are taken in chunks of a fixed size; the part of
// chunk c that lies in sequence b has slot c + b of the workspace (going along
// the tokens one of the two grows from part to part, so no slot is used twice).
struct BalanceGeom {
  int chunk;       // tokens of a chunk
  int64_t chunks;  // ceil(T / chunk)
  int64_t slots;   // chunks + B
  int cols;        // column groups of the join, ceil(E / 16)
  int joins;       // blocks of the join
  // workspace parts, multiples of 16, and the word that counts the join's finished blocks
  size_t sum_bytes, count_bytes, token_bytes;
  size_t bytes() const { return sum_bytes + count_bytes + token_bytes + 16; }
};
BalanceGeom balance_geom(int64_t T, int E, int B);

struct BalanceArgs {
  const void* logits;  // [T, E], fp32 or bf16
  const int64_t* idx;  // [T, K]
  const int32_t* seq;  // [B + 1] or null
  const uint8_t* mask;  // [T] or null
  float* loss;
  int32_t* counts;  // [B, E]
  int32_t* tokens;  // [B]
  float* mean;      // [B, E]
  const float* gloss;
  const void* base;  // backward: the logits' type, or null
  void* glogits;
  int64_t T;
  int E, K, B;
  bool sigmoid, bf16;
  float scale;  // coef * E / (K * B)
  float coef;
  // workspace: by slot, sums [slots, E], counts [slots, E], tokens [slots]; the
  // join's finished blocks
  float* part_sum;
  int32_t* part_count;
  int32_t* part_tokens;
  unsigned* done;
};
hipError_t launch_balance(const BalanceArgs& a, const BalanceGeom& g, hipStream_t s);
hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s);

}  // namespace ep
