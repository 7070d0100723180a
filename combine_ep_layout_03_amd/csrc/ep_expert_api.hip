// C-ABI entry points of ep_mi355x_expert.h: argument checks and error codes.
// Semantics of every call are documented there.
#include "ep_mi355x_expert.h"

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "ep_checks.h"
#include "ep_expert.h"
#include "ep_linear_plan.h"

using namespace ep::checks;

namespace {

static_assert(EP_ACT_NONE == ep::kActNone && EP_ACT_RELU == ep::kActRelu && EP_ACT_SILU == ep::kActSilu &&
                  EP_ACT_GELU == ep::kActGelu && EP_ACT_GELU_TANH == ep::kActGeluTanh,
              "activation numbering");

constexpr int64_t kMaxWidth = 1 << 20;    // W and H
constexpr int64_t kMaxStride = 1 << 21;   // elements: 320 rows stay below 2^32 bytes
constexpr int64_t kMaxGather = 1LL << 36;  // bytes of a gathered token matrix

int width_of(const ep_linear_t* lin) { return lin->gated ? 2 * lin->n_out : lin->n_out; }

// Problem and sizes of both layer calls.
int check_linear(const ep_problem_t* p, const ep_linear_t* lin) {
  const int rc = check_problem(p);
  if (rc != EP_OK) return rc;
  if (p->flags & ~EP_FLAG_GATHER_ROWS) return EP_EINVAL;
  if (!lin || lin->n_out < 1 || lin->activation < EP_ACT_NONE || lin->activation > EP_ACT_GELU_TANH ||
      (lin->gated != 0 && lin->gated != 1))
    return EP_EINVAL;
  if (p->hidden % 8 != 0 || lin->n_out % 8 != 0) return EP_ENOTSUP;
  const int64_t W = lin->gated ? 2LL * lin->n_out : lin->n_out;
  if (p->hidden > kMaxWidth || W > kMaxWidth || W * p->hidden > INT32_MAX) return EP_ENOTSUP;
  // fewer than 2^32 threads in 512 a block, the rounds that a launch is filled up to included
  const int64_t tiles = ep::linear_max_tiles(selections(p), p->num_experts, p->hidden, static_cast<int>(W));
  return tiles < (1 << 22) ? EP_OK : EP_ENOTSUP;
}

int check_stride(const void* p, int64_t stride, int32_t width, int64_t* ld) {
  const int rc = check_rows(p, stride, width, ld);
  return rc != EP_OK ? rc : *ld <= kMaxStride ? EP_OK : EP_EINVAL;
}

// Layout, map and sizes common to both layer calls.
int linear_args(const ep_problem_t* p, const ep_layout_t* L, const ep_linear_t* lin, ep::LinearArgs* a) {
  if (!L || !L->counts || !L->offsets || !L->status) return EP_EINVAL;
  const bool gather = (p->flags & EP_FLAG_GATHER_ROWS) != 0;
  if (gather && (!L->expert_row_src || L->expert_row_capacity < max_rows(p))) return EP_EINVAL;
  a->xmap = gather ? L->expert_row_src : nullptr;
  a->w = static_cast<const uint16_t*>(lin->w);
  a->counts = L->counts;
  a->offsets = L->offsets;
  a->E = p->num_experts;
  a->H = p->hidden;
  a->N = lin->n_out;
  a->W = width_of(lin);
  a->act = lin->activation;
  a->gated = lin->gated != 0;
  a->splits = 1;
  a->status = L->status;
  a->generation = L->generation;
  return EP_OK;
}

bool any_overlap(const Rows& out, std::initializer_list<Rows> others) {
  for (const Rows& r : others)
    if (r.p && rows_overlap(out, r)) return true;
  return false;
}

int check_balance(const ep_balance_t* b) {
  if (!b || b->num_tokens < 0 || b->num_experts < 1 || b->topk < 1 || b->topk > b->num_experts || b->num_seqs < 1)
    return EP_EINVAL;
  if (b->score != EP_SCORE_SOFTMAX && b->score != EP_SCORE_SIGMOID) return EP_EINVAL;
  if (b->logits != EP_LOGITS_FP32 && b->logits != EP_LOGITS_BF16) return EP_EINVAL;
  if (!isfinite(b->coef)) return EP_EINVAL;
  if (b->topk > EP_MAX_TOPK || b->num_experts > EP_MAX_KEYS || b->num_seqs > 65536) return EP_ENOTSUP;
  if (b->num_tokens > INT32_MAX / b->topk) return EP_ENOTSUP;
  return EP_OK;
}

ep::BalanceArgs balance_args(const ep_balance_t* b) {
  ep::BalanceArgs a = {};
  a.T = b->num_tokens;
  a.E = b->num_experts;
  a.K = b->topk;
  a.B = b->num_seqs;
  a.sigmoid = b->score == EP_SCORE_SIGMOID;
  a.bf16 = b->logits == EP_LOGITS_BF16;
  a.coef = b->coef;
  a.scale = static_cast<float>(static_cast<double>(b->coef) * b->num_experts /
                               (static_cast<double>(b->topk) * b->num_seqs));
  return a;
}

}  // namespace

extern "C" {

int ep_expert_linear(const ep_problem_t* p, const ep_layout_t* L, const ep_linear_t* lin,
                     const void* x, int64_t x_row_stride, const void* residual,
                     int64_t residual_row_stride, void* out, int64_t out_row_stride, void* pre,
                     int64_t pre_row_stride, hipStream_t stream) {
  int rc = check_linear(p, lin);
  if (rc != EP_OK) return rc;
  if (p->num_tokens == 0) return EP_OK;
  ep::LinearArgs a = {};
  if ((rc = linear_args(p, L, lin, &a)) != EP_OK) return rc;
  if (!lin->w || !aligned(lin->w, 16) || !aligned(lin->bias, 16)) return EP_EINVAL;
  if ((rc = check_stride(x, x_row_stride, a.H, &a.ldx)) != EP_OK) return rc;
  if ((rc = check_stride(out, out_row_stride, a.N, &a.ldout)) != EP_OK) return rc;
  if (residual && (rc = check_stride(residual, residual_row_stride, a.N, &a.ldres)) != EP_OK) return rc;
  if (pre && (rc = check_stride(pre, pre_row_stride, a.W, &a.ldpre)) != EP_OK) return rc;
  if (a.xmap && p->num_tokens * a.ldx * 2 > kMaxGather) return EP_ENOTSUP;
  const int64_t rows = max_rows(p);
  const Rows rx = {x, a.xmap ? p->num_tokens : rows, 2LL * a.H, 2 * a.ldx};
  const Rows ro = {out, rows, 2LL * a.N, 2 * a.ldout}, rp = {pre, pre ? rows : 0, 2LL * a.W, 2 * a.ldpre};
  const Rows rr = {residual, residual ? rows : 0, 2LL * a.N, 2 * a.ldres};
  const int64_t nw = 2LL * a.E * a.W * a.H, nb = 2LL * a.E * a.W;
  const Rows rw = {lin->w, 1, nw, nw}, rb = {lin->bias, lin->bias ? 1 : 0, nb, nb};
  if (any_overlap(ro, {rx, rw, rb, rp}) || any_overlap(rp, {rx, rw, rb, rr})) return EP_EINVAL;
  if (!(residual == out && a.ldres == a.ldout) && any_overlap(ro, {rr})) return EP_EINVAL;
  a.x = static_cast<const uint16_t*>(x);
  a.bias = static_cast<const uint16_t*>(lin->bias);
  a.res = static_cast<const uint16_t*>(residual);
  a.out = static_cast<uint16_t*>(out);
  a.pre = static_cast<uint16_t*>(pre);
  return ep::launch_linear(a, selections(p), stream) == hipSuccess ? EP_OK : EP_EHIP;
}

size_t ep_expert_linear_workspace_bytes(const ep_problem_t* p, const ep_linear_t* lin) {
  if (check_linear(p, lin) != EP_OK) return 0;
  return ep::linear_geom(selections(p), p->num_experts, p->hidden, width_of(lin)).part_bytes;
}

int ep_expert_linear_backward(const ep_problem_t* p, const ep_layout_t* L, const ep_linear_t* lin,
                              const void* grad_out, int64_t grad_out_row_stride, const void* x,
                              int64_t x_row_stride, const void* pre, int64_t pre_row_stride,
                              void* grad_pre, int64_t grad_pre_row_stride, void* grad_x,
                              int64_t grad_x_row_stride, void* grad_w, void* grad_bias,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_linear(p, lin);
  if (rc != EP_OK) return rc;
  if (grad_bias && !grad_w) return EP_EINVAL;
  if (!aligned(grad_w, 16) || !aligned(grad_bias, 16)) return EP_EINVAL;
  const bool bare = lin->activation == EP_ACT_NONE && !lin->gated;
  ep::LinearArgs a = {};
  if ((rc = linear_args(p, L, lin, &a)) != EP_OK) return rc;
  a.gw = static_cast<uint16_t*>(grad_w);
  a.gb = static_cast<uint16_t*>(grad_bias);
  // no row: the weights' gradients are zero, by the same kernel
  if (p->num_tokens == 0)
    return ep::launch_linear_grads(nullptr, grad_w ? &a : nullptr, 0, stream) == hipSuccess ? EP_OK : EP_EHIP;
  int64_t ldgo = 0;
  if ((rc = check_stride(grad_out, grad_out_row_stride, a.N, &ldgo)) != EP_OK) return rc;
  if (grad_w && (rc = check_stride(x, x_row_stride, a.H, &a.ldx)) != EP_OK) return rc;
  if (grad_x && (!lin->w || !aligned(lin->w, 16))) return EP_EINVAL;
  if (grad_x && (rc = check_stride(grad_x, grad_x_row_stride, a.H, &a.ldout)) != EP_OK) return rc;
  ep::ActBackwardArgs b = {};
  if (bare) {
    if (pre || grad_pre) return EP_EINVAL;
  } else {
    if ((rc = check_stride(pre, pre_row_stride, a.W, &b.ldpre)) != EP_OK) return rc;
    if ((rc = check_stride(grad_pre, grad_pre_row_stride, a.W, &b.ldgpre)) != EP_OK) return rc;
  }
  if (a.xmap && grad_w && p->num_tokens * a.ldx * 2 > kMaxGather) return EP_ENOTSUP;
  const int64_t rows = max_rows(p);
  const ep::LinearGeom g = ep::linear_geom(selections(p), a.E, a.H, a.W);
  const int64_t nw = 2LL * a.E * a.W * a.H, nb = 2LL * a.E * a.W;
  const Rows ro = {grad_out, rows, 2LL * a.N, 2 * ldgo};
  const Rows rx = {grad_w ? x : nullptr, a.xmap ? p->num_tokens : rows, 2LL * a.H, 2 * a.ldx};
  const Rows rw = {grad_x ? lin->w : nullptr, 1, nw, nw};
  const Rows rp = {pre, pre ? rows : 0, 2LL * a.W, 2 * b.ldpre};
  const Rows gp = {grad_pre, grad_pre ? rows : 0, 2LL * a.W, 2 * b.ldgpre};
  const Rows gx = {grad_x, grad_x ? rows : 0, 2LL * a.H, 2 * a.ldout};
  const Rows gw = {grad_w, grad_w ? 1 : 0, nw, nw}, gb = {grad_bias, grad_bias ? 1 : 0, nb, nb};
  if (any_overlap(gp, {ro, rx, rw, gx, gw, gb}) || any_overlap(gx, {ro, rx, rw, rp, gw, gb}) ||
      any_overlap(gw, {ro, rx, rw, rp, gb}) || any_overlap(gb, {ro, rx, rw, rp}))
    return EP_EINVAL;
  if (!(pre == grad_pre && b.ldpre == b.ldgpre) && any_overlap(gp, {rp})) return EP_EINVAL;
  if (grad_w) {  // nothing else uses it
    if (!workspace || !aligned(workspace, 16)) return EP_EINVAL;
    if (workspace_bytes < g.part_bytes) return EP_EWORKSPACE;
    if (workspace_overlaps(workspace, g.part_bytes, {ro, rx, rw, rp, gp, gx, gw, gb})) return EP_EINVAL;
  }
  a.x = static_cast<const uint16_t*>(x);
  if (bare) {
    a.g = static_cast<const uint16_t*>(grad_out);
    a.ldg = ldgo;
  } else {
    b.go = static_cast<const uint16_t*>(grad_out);
    b.ldgo = ldgo;
    b.pre = static_cast<const uint16_t*>(pre);
    b.gpre = static_cast<uint16_t*>(grad_pre);
    b.counts = a.counts;
    b.offsets = a.offsets;
    b.E = a.E;
    b.N = a.N;
    b.act = a.act;
    b.gated = a.gated;
    b.padded = p->expert_alignment > 1;
    b.status = a.status;
    b.generation = a.generation;
    if (ep::launch_act_backward(b, rows, stream) != hipSuccess) return EP_EHIP;
    a.g = static_cast<const uint16_t*>(grad_pre);
    a.ldg = b.ldgpre;
  }
  ep::LinearArgs ax = a;
  ax.out = static_cast<uint16_t*>(grad_x);
  a.splits = g.splits;
  a.part = static_cast<float*>(workspace);
  return ep::launch_linear_grads(grad_x ? &ax : nullptr, grad_w ? &a : nullptr, selections(p), stream) == hipSuccess
             ? EP_OK
             : EP_EHIP;
}

size_t ep_balance_workspace_bytes(const ep_balance_t* b) {
  if (check_balance(b) != EP_OK) return 0;
  return ep::balance_geom(b->num_tokens, b->num_experts, b->num_seqs).bytes();
}

int ep_balance_loss(const ep_balance_t* b, const void* logits, const int64_t* topk_idx,
                    const int32_t* seq_offsets, const uint8_t* token_mask, float* loss,
                    int32_t* counts, int32_t* tokens, float* mean, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_balance(b);
  if (rc != EP_OK) return rc;
  if (!loss || !counts || !tokens || !mean || (!seq_offsets && b->num_seqs != 1)) return EP_EINVAL;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(mean, 4) || !aligned(seq_offsets, 4))
    return EP_EINVAL;
  ep::BalanceArgs a = balance_args(b);
  const ep::BalanceGeom g = ep::balance_geom(a.T, a.E, a.B);
  const int el = a.bf16 ? 2 : 4;
  if (a.T > 0 && (!logits || !topk_idx || !aligned(logits, el) || !aligned(topk_idx, 8))) return EP_EINVAL;
  const int64_t be = 4LL * a.B * a.E;
  const bool some = a.T > 0;
  const Span sl = {some ? logits : nullptr, a.T * a.E * el}, si = {some ? topk_idx : nullptr, 8 * a.T * a.K};
  const Span sm = {some ? token_mask : nullptr, a.T}, ss = {seq_offsets, 4LL * (a.B + 1)};
  if (some) {
    if (!workspace || !aligned(workspace, 16)) return EP_EINVAL;
    if (workspace_bytes < g.bytes()) return EP_EWORKSPACE;
  }
  if (clash({{loss, 4}, {counts, be}, {tokens, 4LL * a.B}, {mean, be},
             {some ? workspace : nullptr, static_cast<int64_t>(g.bytes())}},
            {sl, si, sm, ss}))
    return EP_EINVAL;
  a.logits = logits;
  a.idx = topk_idx;
  a.seq = seq_offsets;
  a.mask = token_mask;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.mean = mean;
  char* ws = static_cast<char*>(workspace);
  auto part = [&](size_t bytes) {
    char* at = ws;
    ws += bytes;
    return at;
  };
  if (some) {
    a.part_sum = reinterpret_cast<float*>(part(g.sum_bytes));
    a.part_count = reinterpret_cast<int32_t*>(part(g.count_bytes));
    a.part_tokens = reinterpret_cast<int32_t*>(part(g.token_bytes));
    a.done = reinterpret_cast<unsigned*>(ws);
  }
  return ep::launch_balance(a, g, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

int ep_balance_loss_backward(const ep_balance_t* b, const float* grad_loss, const void* logits,
                             const int32_t* seq_offsets, const uint8_t* token_mask,
                             const int32_t* counts, const int32_t* tokens, const void* grad_base,
                             void* grad_logits, hipStream_t stream) {
  const int rc = check_balance(b);
  if (rc != EP_OK) return rc;
  if (!seq_offsets && b->num_seqs != 1) return EP_EINVAL;
  if (b->num_tokens == 0) return EP_OK;
  if (!grad_loss || !logits || !counts || !tokens || !grad_logits) return EP_EINVAL;
  ep::BalanceArgs a = balance_args(b);
  const int el = a.bf16 ? 2 : 4;
  if (!aligned(grad_loss, 4) || !aligned(logits, el) || !aligned(seq_offsets, 4) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(grad_base, el) || !aligned(grad_logits, el))
    return EP_EINVAL;
  const int64_t bytes = a.T * a.E * el;
  if (clash({{grad_logits, bytes}},
            {{grad_loss, 4}, {logits, bytes}, {seq_offsets, 4LL * (a.B + 1)}, {token_mask, a.T},
             {counts, 4LL * a.B * a.E}, {tokens, 4LL * a.B}, {grad_base == grad_logits ? nullptr : grad_base, bytes}}))
    return EP_EINVAL;
  a.gloss = grad_loss;
  a.logits = logits;
  a.seq = seq_offsets;
  a.mask = token_mask;
  a.counts = const_cast<int32_t*>(counts);  // read only
  a.tokens = const_cast<int32_t*>(tokens);  // read only
  a.base = grad_base;
  a.glogits = grad_logits;
  return ep::launch_balance_backward(a, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

}  // extern "C"
