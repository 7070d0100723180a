/*
 * ep_mi355x_layer.h — C ABI of the operators around the token dispatch and
 * combine of ep_mi355x.h: the router that makes the selections, the gradients
 * of router and combine, and low-rank adapters over the layout's segments.
 *
 * Not from the pages: operators of this library, defined by the formulas
 * below.  The conventions, return codes, status words and the structs
 * ep_problem_t and ep_layout_t are those of ep_mi355x.h.
 */
#ifndef EP_MI355X_LAYER_H
#define EP_MI355X_LAYER_H

#include "ep_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- limits ----------------------------------------------------------- */
#define EP_MAX_ROUTE_GROUPS 64 /* expert groups of a group-limited router */
#define EP_MAX_LORA_RANK 128

/* ---- router ----------------------------------------------------------- */
#define EP_SCORE_SOFTMAX 0 /* s[t,e] = exp(l[t,e]) / sum_e' exp(l[t,e']) */
#define EP_SCORE_SIGMOID 1 /* s[t,e] = 1 / (1 + exp(-l[t,e])) */

#define EP_LOGITS_FP32 0
#define EP_LOGITS_BF16 1

/* A router.
 *   num_tokens   T >= 0, T * K < 2^31
 *   num_experts  E in [1, EP_MAX_KEYS]
 *   topk         K in [1, EP_MAX_TOPK], K <= E
 *   score, logits  EP_SCORE_*, EP_LOGITS_*
 *   num_groups   0 = every expert may be chosen; G in [1, EP_MAX_ROUTE_GROUPS]
 *                dividing E = the experts form G contiguous groups and only
 *                topk_groups of them may be chosen from
 *   topk_groups  with groups, in [1, G]; K <= topk_groups * E / G
 *   group_top    a group's value is the sum of its group_top largest
 *                selection values: 1 or 2
 *   renormalize  0 or 1: the chosen scores are divided by their sum
 *   scale        factor on the weights (finite) */
typedef struct ep_router {
  int64_t num_tokens;
  int32_t num_experts;
  int32_t topk;
  int32_t score;
  int32_t logits;
  int32_t num_groups;
  int32_t topk_groups;
  int32_t group_top;
  int32_t renormalize;
  float scale;
} ep_router_t;

/* Routing: topk_idx int64 [T*K] and topk_weights fp32 [T*K], the inputs of
 * ep_layout and ep_combine, from logits [T*E] (fp32 or bf16, row-major).
 *
 * An expert's selection value is s[t,e] + bias[e] (bias fp32 [E], a balance
 * bias that takes part in the choice and not in the weights), or without a
 * bias (NULL) the logit itself, which orders the experts as either score
 * does.  With groups, a group's value is the sum of its group_top largest
 * selection values (group_top == 2 without a bias: of its largest scores)
 * and the topk_groups groups of largest value stay open.  The K experts of
 * largest selection value in the open groups are chosen, in descending
 * order.  Equal values, of groups or experts, go to the lowest index.
 * Selection values are compared as if computed in binary64.
 *
 * An expert whose logit is NaN or -inf, or whose bias is NaN or -inf, cannot
 * be chosen (nor does it count in the softmax, if its logit is the reason); a
 * logit of +inf counts as the largest finite fp32.  token_mask (uint8 [T],
 * may be NULL): a token whose byte is 0 gets no selection.  Entries without
 * an expert to choose are -1 with weight 0, and come last.
 *
 * topk_weights[t,k] = scale * s[t, topk_idx[t,k]], with renormalize divided
 * by the token's sum of chosen scores (formed relative to the largest, so
 * that scores which underflow still share it), in fp32.
 * logits, bias and topk_weights must be aligned to their elements, topk_idx
 * to 8 bytes; the outputs must overlap neither an input nor each other. */
int ep_route(const ep_router_t* r, const void* logits, const float* bias,
             const uint8_t* token_mask, int64_t* topk_idx, float* topk_weights,
             hipStream_t stream);

/* Gradient of ep_route's weights: grad_logits[t,e] (the logits' type, every
 * element written) = sum_k grad_weights[t,k] * d topk_weights[t,k] /
 * d logits[t,e], for the selections topk_idx [T*K] that ep_route returned.
 * With s the scores, g = scale * grad_weights and w the chosen scores over
 * their sum:
 *   softmax:              s_e * (g_e - sum_k g_k s_k)
 *   softmax, renormalize: w_k * (g_k - sum_j g_j w_j) at e = topk_idx[t,k], else 0
 *   sigmoid:              g_k * s_k * (1 - s_k) there, else 0
 *   sigmoid, renormalize: w_k * (1 - s_k) * (g_k - sum_j g_j w_j) there, else 0
 * The choice is constant and the bias has no gradient.  Entries of topk_idx
 * outside [0, E) have no part; an expert named twice gets both terms.  Sums
 * are fp32; a bf16 result is rounded once.  grad_logits must not overlap an
 * input.  r's groups are not used and may be 0. */
int ep_route_backward(const ep_router_t* r, const void* logits, const int64_t* topk_idx,
                      const float* grad_weights, void* grad_logits, hipStream_t stream);

/* ---- gradient of ep_combine ------------------------------------------- */
/* For every valid selection (t,k) with slot r = slot[t,k] < y_rows:
 *   grad_y[r, h]       = bf16_rne( topk_weights[t,k] * grad_out[t, h] )
 *   grad_weights[t, k] = sum_h grad_out[t, h] * y[r, h]     (fp32)
 * and grad_weights[t,k] = 0 for the others; a slot >= y_rows also sets
 * EP_STATUS_COMBINE_OOB.  grad_out bf16 [T*H], y and grad_y bf16 [y_rows*H]
 * in expert-major receive order; rows of grad_y that no selection owns are
 * not written.  Both combine orders have this gradient; a bias row's gradient
 * is grad_out itself.  Each product of grad_y is one fp32 rounding before the
 * bf16 one; the sum runs in fp32 in a fixed order, so equal inputs give equal
 * bytes.  The outputs must overlap neither an input nor each other.  A stale L
 * writes nothing but EP_STATUS_STALE = 1.
 * (The gradient of ep_dispatch is ep_combine with unit weights.) */
int ep_combine_backward(const ep_problem_t* p, const ep_layout_t* L, const float* topk_weights,
                        const void* grad_out, const void* y, int64_t y_rows, void* grad_y,
                        float* grad_weights, hipStream_t stream);

/* ---- low-rank adapters ------------------------------------------------ */
#define EP_LORA_SCATTER_ROWS 1 /* base and out rows are token rows */

/* Adapters, one per expert of the layout (for requests with adapters of
 * their own, the layout of topk_idx = adapter id per token, K = 1).
 *   a       bf16 [E, R, H], b bf16 [E, N, R], 16-byte aligned
 *   scales  fp32 [E], or NULL for 1
 *   rank    R, a multiple of 8 in [8, EP_MAX_LORA_RANK]
 *   n_out   N, a multiple of 8
 *   flags   EP_LORA_SCATTER_ROWS or 0 */
typedef struct ep_lora_weights {
  const void* a;
  const void* b;
  const float* scales;
  int32_t rank;
  int32_t n_out;
  int32_t flags;
} ep_lora_weights_t;

/* Bytes of device workspace ep_lora (backward == 0) or ep_lora_backward (1)
 * needs for this problem; 0 if ep_lora would refuse it.  Host only.  The backward
 * pass keeps partial gradients of R * (H + N) fp32 each: up to 64 for T * K (and
 * padding) up to 131,072 rows, one for 2048 rows above. */
size_t ep_lora_workspace_bytes(const ep_problem_t* p, const ep_lora_weights_t* w, int32_t backward);

/* out = base + scales[e] * (x A_e^T) B_e^T over the expert-major segments: for
 * every expert e and row r in [offsets[e], offsets[e] + counts[e]),
 *   out[o(r), n] = bf16_rne( base[o(r), n] +
 *                  scales[e] * sum_j b[e,n,j] * (sum_h a[e,j,h] * x[i(r), h]) )
 * where i(r) = r, or expert_row_src[r] with EP_FLAG_GATHER_ROWS in p->flags
 * (x is the token matrix, as in ep_expert_gemm), and o(r) = r, or
 * expert_row_src[r] with EP_LORA_SCATTER_ROWS (needs K = 1: each token row
 * has one owner).  The inner product is held in fp32 and enters the outer one
 * unrounded; sums are fp32.  Infinities and NaN go where the formula takes
 * them (an inner product below 2^-133 counts as 0 beside an infinity).
 *   x     bf16, row stride x_row_stride elements (0 = H)
 *   base  bf16, row stride base_row_stride (0 = N); NULL = zeros; may be out
 *         itself (same pointer and stride: the delta is added in place)
 *   out   bf16, row stride out_row_stride (0 = N)
 * Rows of no selection: with EP_LORA_SCATTER_ROWS they become base's row
 * (zeros without one), so all T rows of out are defined; otherwise they are
 * not written.  out must not overlap x, nor base unless it is base (token
 * matrices have T rows, the others are taken to have T * K + E * (A - 1), A the
 * alignment or 1).
 * Requires H % 8 == 0, row strides multiples of 8, bases 16-byte aligned
 * (EP_ENOTSUP for sizes, EP_EINVAL for strides and bases), and `workspace`
 * of ep_lora_workspace_bytes, 16-byte aligned (contents need no
 * initialisation and are clobbered; it must not overlap another argument, and
 * calls that may overlap in time need their own).  A stale L writes no row and sets EP_STATUS_STALE. */
int ep_lora(const ep_problem_t* p, const ep_layout_t* L, const ep_lora_weights_t* w, const void* x,
            int64_t x_row_stride, const void* base, int64_t base_row_stride, void* out,
            int64_t out_row_stride, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradients of ep_lora for grad_out (bf16, rows as out's: o(r)), with
 * u_r = A_e x[i(r)] and v_r = B_e^T grad_out[o(r)]:
 *   grad_x[o(r)] = bf16_rne( grad_base[o(r)] + scales[e] * A_e^T v_r )
 *   grad_a[e]    = bf16_rne( scales[e] * sum_r v_r x[i(r)]^T )       [E, R, H]
 *   grad_b[e]    = bf16_rne( scales[e] * sum_r grad_out[o(r)] u_r^T ) [E, N, R]
 * grad_x's rows follow out (with K > 1 and gathered rows each receive row
 * keeps its own; ep_combine with unit weights adds a token's).  grad_base
 * (bf16, NULL = zeros, may be grad_x itself) is the gradient that the
 * projection beside the adapter sends to x.  Rows of no selection are treated
 * as ep_lora treats out's.  Every element of grad_a and grad_b is written, 0
 * for an expert without rows.  u and v are held in fp32 and enter the products
 * unrounded; sums are fp32 in a fixed order.  Row strides are as in
 * ep_lora (0 = H for x, grad_base and grad_x, N for grad_out), as are the
 * checks. */
int ep_lora_backward(const ep_problem_t* p, const ep_layout_t* L, const ep_lora_weights_t* w,
                     const void* grad_out, int64_t grad_out_row_stride, const void* x,
                     int64_t x_row_stride, const void* grad_base, int64_t grad_base_row_stride,
                     void* grad_x, int64_t grad_x_row_stride, void* grad_a, void* grad_b,
                     void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_MI355X_LAYER_H */
