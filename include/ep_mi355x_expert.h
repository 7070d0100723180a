/*
 * ep_mi355x_expert.h — C ABI of the experts' layers over the segments of
 * ep_mi355x.h: the grouped product with bias, activation and residual in its
 * epilogue, its gradients, and the balance loss of the router that feeds it.
 *
 * Not from the pages: operators of this library, defined by the formulas
 * below.  The conventions, return codes, status words and the structs
 * ep_problem_t and ep_layout_t are those of ep_mi355x.h, EP_SCORE_* and
 * EP_LOGITS_* those of ep_mi355x_layer.h.
 */
#ifndef EP_MI355X_EXPERT_H
#define EP_MI355X_EXPERT_H

#include "ep_mi355x_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- an expert's layer ------------------------------------------------- */
#define EP_ACT_NONE 0      /* z */
#define EP_ACT_RELU 1      /* max(z, 0); derivative 0 at 0 */
#define EP_ACT_SILU 2      /* z / (1 + exp(-z)) */
#define EP_ACT_GELU 3      /* z (1 + erf(z / sqrt 2)) / 2 */
#define EP_ACT_GELU_TANH 4 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */

/* The experts' weights and what follows their product.
 *   w       bf16 [E, W, H], 16-byte aligned; H is the problem's hidden
 *   bias    bf16 [E, W], 16-byte aligned, or NULL for none
 *   n_out   N, a multiple of 8: columns of the result
 *   activation  EP_ACT_*
 *   gated   0: W = N; 1: W = 2 N, rows [0, N) of an expert's weights are the
 *           gate's and rows [N, 2 N) what it multiplies */
typedef struct ep_linear {
  const void* w;
  const void* bias;
  int32_t n_out;
  int32_t activation;
  int32_t gated;
} ep_linear_t;

/* For every expert e and row r in [offsets[e], offsets[e] + counts[e]):
 *   z[n]      = sum_h x[i(r), h] * w[e, n, h] + bias[e, n],  n < W
 *   pre[r, n] = bf16_rne( z[n] )                              (if pre is given)
 *   out[r, n] = bf16_rne( act(z[n]) + residual[r, n] ),       n < N, or gated
 *   out[r, n] = bf16_rne( act(z[n]) * z[N + n] + residual[r, n] )
 * where i(r) = r, or expert_row_src[r] with EP_FLAG_GATHER_ROWS in p->flags (x
 * is the token matrix, as in ep_expert_gemm).  Sums, activation and residual
 * are fp32, the activation of the unrounded z.  Infinities and NaN go where
 * the formulas take them, row by row.
 *   x         bf16, row stride x_row_stride elements (0 = H)
 *   residual  bf16, row stride residual_row_stride (0 = N); NULL = none; may be
 *             out itself (same pointer and stride)
 *   out       bf16, row stride out_row_stride (0 = N)
 *   pre       bf16, row stride pre_row_stride (0 = W), or NULL; what the
 *             gradient needs
 * Rows of no selection are not written.  Neither out nor pre may overlap
 * another argument (but out residual, as above; rows are taken to be T for
 * gathered x, T * K + E * (A - 1) otherwise, A the alignment or 1).
 * Requires H % 8 == 0, N % 8 == 0, row strides multiples of 8 up to 2^21,
 * bases 16-byte aligned, W and H up to 2^20 with W * H < 2^31, fewer than
 * 2^22 tiles of 128 rows x 128 columns (of the T * K selections; padding counts
 * in no tile) and, with gathered rows, x of 64 GiB at most (EP_ENOTSUP for
 * sizes, EP_EINVAL for strides and bases).  Other flags than
 * EP_FLAG_GATHER_ROWS are refused.  A stale L writes nothing but
 * EP_STATUS_STALE = 1. */
int ep_expert_linear(const ep_problem_t* p, const ep_layout_t* L, const ep_linear_t* lin,
                     const void* x, int64_t x_row_stride, const void* residual,
                     int64_t residual_row_stride, void* out, int64_t out_row_stride, void* pre,
                     int64_t pre_row_stride, hipStream_t stream);

/* Bytes of device workspace ep_expert_linear_backward needs for this problem
 * (partial weight gradients, where experts are few); 0 if it would refuse the
 * sizes.  Host only. */
size_t ep_expert_linear_workspace_bytes(const ep_problem_t* p, const ep_linear_t* lin);

/* Gradients of ep_expert_linear for grad_out (bf16, rows as out's).  With z =
 * pre[r] as the forward call rounded it,
 *   grad_pre[r, n]     = bf16_rne( grad_out[r, n] * act'(z[n]) ),  or gated
 *   grad_pre[r, n]     = bf16_rne( grad_out[r, n] * z[N + n] * act'(z[n]) )
 *   grad_pre[r, N + n] = bf16_rne( grad_out[r, n] * act(z[n]) )
 *   grad_x[r, h]    = bf16_rne( sum_n grad_pre[r, n] * w[e, n, h] )
 *   grad_w[e, n, h] = bf16_rne( sum_r grad_pre[r, n] * x[i(r), h] )
 *   grad_bias[e, n] = bf16_rne( sum_r grad_pre[r, n] )
 * sums in fp32 in a fixed order, so equal inputs give equal bytes.  Without
 * activation and gate grad_pre is grad_out itself: pre and grad_pre are NULL.
 * The gradient of the residual is grad_out itself.
 *   grad_out   bf16, row stride grad_out_row_stride (0 = N)
 *   x, pre     as in the forward call
 *   grad_pre   bf16, row stride grad_pre_row_stride (0 = W); may be pre
 *              itself (same pointer and stride)
 *   grad_x     bf16 receive rows (with gathered rows each keeps its own;
 *              ep_combine with unit weights adds a token's), row stride
 *              grad_x_row_stride (0 = H), or NULL to leave it out
 *   grad_w     bf16 [E, W, H], 16-byte aligned, or NULL
 *   grad_bias  bf16 [E, W], 16-byte aligned, or NULL
 * grad_bias needs grad_w; x may be NULL without grad_w.  Every element of
 * grad_w and grad_bias is written, 0 for an expert without rows; rows of
 * grad_pre and grad_x of no selection are not written.  lin->bias is not read.
 * Limits as in ep_expert_linear; the outputs must overlap neither an input nor
 * each other.  `workspace` of ep_expert_linear_workspace_bytes, 16-byte
 * aligned (its contents need no initialisation and are clobbered; calls that
 * may overlap in time need their own); not used, and may be NULL, without
 * grad_w. */
int ep_expert_linear_backward(const ep_problem_t* p, const ep_layout_t* L, const ep_linear_t* lin,
                              const void* grad_out, int64_t grad_out_row_stride, const void* x,
                              int64_t x_row_stride, const void* pre, int64_t pre_row_stride,
                              void* grad_pre, int64_t grad_pre_row_stride, void* grad_x,
                              int64_t grad_x_row_stride, void* grad_w, void* grad_bias,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- balance loss ------------------------------------------------------ */
/* A balance loss over sequences of tokens.
 *   num_tokens   T >= 0, T * K < 2^31
 *   num_experts  E in [1, EP_MAX_KEYS]
 *   topk         K in [1, EP_MAX_TOPK]
 *   score, logits  EP_SCORE_*, EP_LOGITS_*
 *   num_seqs     B in [1, 65536]
 *   coef         factor of the loss (finite)
 * Sequence b is the tokens [seq_offsets[b], seq_offsets[b + 1]) (int32 [B + 1],
 * device, ascending, within [0, T]; tokens before the first and from the last
 * on belong to none), or, with seq_offsets NULL and B = 1, all of them. */
typedef struct ep_balance {
  int64_t num_tokens;
  int32_t num_experts;
  int32_t topk;
  int32_t score;
  int32_t logits;
  int32_t num_seqs;
  float coef;
} ep_balance_t;

/* Bytes of device workspace ep_balance_loss needs; 0 if it would refuse the
 * sizes.  Host only. */
size_t ep_balance_workspace_bytes(const ep_balance_t* b);

/* With p[t] the scores of token t over their sum (softmax: themselves), n_b
 * the tokens of sequence b whose byte of token_mask (uint8 [T], may be NULL)
 * is not 0, and all sums over those tokens:
 *   tokens[b]    = n_b
 *   counts[b, e] = selections (t, k) with topk_idx[t, k] = e
 *   mean[b, e]   = sum_t p[t, e] / n_b                    (0 if n_b = 0)
 *   loss[0]      = coef / B * sum_b E / (K n_b) * sum_e counts[b, e] mean[b, e]
 * A sequence without tokens adds 0.  logits [T, E] as in ep_route: a NaN or
 * -inf logit takes an expert out of its token (p = 0; all out: the token's p
 * is 0, and it counts in n_b), +inf counts as the largest finite fp32.  Ids
 * outside [0, E) are not counted.  loss fp32 [1], counts int32 [B, E], tokens
 * int32 [B], mean fp32 [B, E], every element written; sums in fixed order, so
 * equal inputs give equal bytes.  Offsets that descend or leave [0, T] give
 * values of no meaning, and no access out of range.  The outputs and the
 * workspace (16-byte aligned, contents need no initialisation; calls that may
 * overlap in time need their own) must not overlap another argument. */
int ep_balance_loss(const ep_balance_t* b, const void* logits, const int64_t* topk_idx,
                    const int32_t* seq_offsets, const uint8_t* token_mask, float* loss,
                    int32_t* counts, int32_t* tokens, float* mean, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);

/* Gradient of loss to the logits: with f[e] = grad_loss[0] * coef * E *
 * counts[b, e] / (B * K * n_b^2) for the sequence b of token t,
 *   softmax:  grad_logits[t, e] = p_e (f_e - sum_j f_j p_j)           + grad_base[t, e]
 *   sigmoid:  grad_logits[t, e] = p_e (1 - s_e) (f_e - sum_j f_j p_j) + grad_base[t, e]
 * in the logits' type, every element written; a token that its mask or the
 * sequences leave out gets grad_base alone, as does an expert that its logit
 * takes out.  counts (int32 [B, E]) and tokens (int32 [B]) as ep_balance_loss
 * wrote them; the counts are constants.  grad_base (the logits' type, NULL =
 * zeros, may be grad_logits itself) is the gradient that comes to the logits
 * another way, such as ep_route_backward's.  grad_logits must not overlap
 * another argument but grad_base. */
int ep_balance_loss_backward(const ep_balance_t* b, const float* grad_loss, const void* logits,
                             const int32_t* seq_offsets, const uint8_t* token_mask,
                             const int32_t* counts, const int32_t* tokens, const void* grad_base,
                             void* grad_logits, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_MI355X_EXPERT_H */
