// C-ABI entry points of ep_mi355x_layer.h: argument checks and error codes.
// Semantics of every call are documented there.
#include "ep_mi355x_layer.h"

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "ep_checks.h"
#include "ep_layer.h"

using namespace ep::checks;

namespace {

static_assert(EP_STATUS_COMBINE_OOB == ep::kStatusCombineOob, "status word numbering");
static_assert(EP_MAX_ROUTE_GROUPS == ep::kMaxRouteGroups, "route group limit");

int check_router(const ep_router_t* r, bool groups) {
  if (!r || r->num_tokens < 0 || r->num_experts < 1 || r->topk < 1 || r->topk > r->num_experts)
    return EP_EINVAL;
  if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_EINVAL;
  if (r->logits != EP_LOGITS_FP32 && r->logits != EP_LOGITS_BF16) return EP_EINVAL;
  if ((r->renormalize != 0 && r->renormalize != 1) || !isfinite(r->scale)) return EP_EINVAL;
  if (r->topk > EP_MAX_TOPK || r->num_experts > EP_MAX_KEYS) return EP_ENOTSUP;
  if (r->num_tokens > INT32_MAX / r->topk) return EP_ENOTSUP;  // what ep_layout takes
  if (groups && r->num_groups != 0) {
    if (r->num_groups < 0 || r->num_experts % r->num_groups != 0) return EP_EINVAL;
    if (r->topk_groups < 1 || r->topk_groups > r->num_groups) return EP_EINVAL;
    if (r->group_top != 1 && r->group_top != 2) return EP_EINVAL;
    if (r->topk > r->topk_groups * (r->num_experts / r->num_groups)) return EP_EINVAL;
    if (r->num_groups > EP_MAX_ROUTE_GROUPS) return EP_ENOTSUP;
  }
  return EP_OK;
}

ep::LoraGeom geom_of(const ep_problem_t* p, const ep_lora_weights_t* w, bool backward) {
  return ep::lora_geom(max_rows(p), p->num_experts, p->hidden, w->n_out, w->rank, backward);
}

// Problem, adapters and sizes of both adapter calls.
int check_lora(const ep_problem_t* p, const ep_lora_weights_t* w) {
  const int rc = check_problem(p);
  if (rc != EP_OK) return rc;
  if (!w || w->rank < 1 || w->n_out < 1 || (w->flags & ~EP_LORA_SCATTER_ROWS)) return EP_EINVAL;
  if ((w->flags & EP_LORA_SCATTER_ROWS) && p->topk != 1) return EP_EINVAL;
  if (p->hidden % 8 != 0 || w->n_out % 8 != 0 || w->rank % 8 != 0 || w->rank > EP_MAX_LORA_RANK)
    return EP_ENOTSUP;
  // grid limits: fewer than 2^32 threads, and 2^31 row indices (check_problem)
  if (static_cast<int64_t>(p->hidden) + w->n_out > (1 << 24)) return EP_ENOTSUP;
  const ep::LoraGeom g = geom_of(p, w, true);
  const int64_t cols = (p->hidden > w->n_out ? p->hidden : w->n_out) / 512 + 1;
  if (g.max_tiles >= (1 << 23) ||
      g.max_expand * cols + ep::kLoraMaxCopyBlocks + ep::lora_weight_blocks(g, p->hidden, w->n_out, w->rank) >=
          (1 << 24))
    return EP_ENOTSUP;
  return EP_OK;
}

// Layout, maps and adapters common to both adapter calls.
int lora_args(const ep_problem_t* p, const ep_layout_t* L, const ep_lora_weights_t* w, ep::LoraArgs* a) {
  if (!L || !L->counts || !L->offsets || !L->status || (p->num_tokens > 0 && !L->slot)) return EP_EINVAL;
  if (!w->a || !w->b || !aligned(w->a, 16) || !aligned(w->b, 16) || !aligned(w->scales, 4)) return EP_EINVAL;
  const bool gather = (p->flags & EP_FLAG_GATHER_ROWS) != 0;
  const bool scatter = (w->flags & EP_LORA_SCATTER_ROWS) != 0;
  if ((gather || scatter) && (!L->expert_row_src || L->expert_row_capacity < max_rows(p))) return EP_EINVAL;
  a->xmap = gather ? L->expert_row_src : nullptr;
  a->omap = scatter ? L->expert_row_src : nullptr;
  a->a = static_cast<const uint16_t*>(w->a);
  a->b = static_cast<const uint16_t*>(w->b);
  a->scales = w->scales;
  a->counts = L->counts;
  a->offsets = L->offsets;
  a->slot = L->slot;
  a->T = p->num_tokens;
  a->K = p->topk;
  a->E = p->num_experts;
  a->H = p->hidden;
  a->N = w->n_out;
  a->R = w->rank;
  a->status = L->status;
  a->generation = L->generation;
  return EP_OK;
}

void set_workspace(ep::LoraArgs* a, const ep::LoraGeom& g, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  auto part = [&](size_t bytes) {
    char* at = ws;
    ws += bytes;
    return at;
  };
  a->expand_tiles = reinterpret_cast<int32_t*>(part(g.expand_bytes));
  a->chunks = reinterpret_cast<int32_t*>(part(g.chunk_bytes));
  a->u = reinterpret_cast<float*>(part(g.u_bytes));
  a->v = reinterpret_cast<float*>(part(g.v_bytes));
  a->slots = reinterpret_cast<float*>(part(g.slot_bytes));
}

ep::RouteArgs route_args(const ep_router_t* r) {
  ep::RouteArgs a = {};
  a.T = r->num_tokens;
  a.E = r->num_experts;
  a.K = r->topk;
  a.sigmoid = r->score == EP_SCORE_SIGMOID;
  a.renorm = r->renormalize != 0;
  a.bf16 = r->logits == EP_LOGITS_BF16;
  a.scale = r->scale;
  return a;
}

}  // namespace

extern "C" {

int ep_route(const ep_router_t* r, const void* logits, const float* bias,
             const uint8_t* token_mask, int64_t* topk_idx, float* topk_weights,
             hipStream_t stream) {
  const int rc = check_router(r, true);
  if (rc != EP_OK) return rc;
  if (r->num_tokens == 0) return EP_OK;
  if (!logits || !topk_idx || !topk_weights) return EP_EINVAL;
  const int el = r->logits == EP_LOGITS_FP32 ? 4 : 2;
  if (!aligned(logits, el) || !aligned(bias, 4) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4))
    return EP_EINVAL;
  const int64_t sel = r->num_tokens * r->topk;
  if (clash({{topk_idx, 8 * sel}, {topk_weights, 4 * sel}},
            {{logits, r->num_tokens * r->num_experts * el}, {bias, 4LL * r->num_experts}, {token_mask, r->num_tokens}}))
    return EP_EINVAL;
  ep::RouteArgs a = route_args(r);
  a.logits = logits;
  a.bias = bias;
  a.mask = token_mask;
  a.idx = topk_idx;
  a.w = topk_weights;
  a.G = r->num_groups;
  a.gsize = a.G ? a.E / a.G : a.E;
  a.tg = r->topk_groups;
  a.gtop = r->group_top;
  return ep::launch_route(a, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

int ep_route_backward(const ep_router_t* r, const void* logits, const int64_t* topk_idx,
                      const float* grad_weights, void* grad_logits, hipStream_t stream) {
  const int rc = check_router(r, false);
  if (rc != EP_OK) return rc;
  if (r->num_tokens == 0) return EP_OK;
  if (!logits || !topk_idx || !grad_weights || !grad_logits) return EP_EINVAL;
  const int el = r->logits == EP_LOGITS_FP32 ? 4 : 2;
  if (!aligned(logits, el) || !aligned(grad_logits, el) || !aligned(topk_idx, 8) ||
      !aligned(grad_weights, 4))
    return EP_EINVAL;
  const int64_t bytes = r->num_tokens * r->num_experts * el;
  const int64_t sel = r->num_tokens * r->topk;
  if (clash({{grad_logits, bytes}}, {{logits, bytes}, {topk_idx, 8 * sel}, {grad_weights, 4 * sel}})) return EP_EINVAL;
  ep::RouteArgs a = route_args(r);
  a.logits = logits;
  a.idx = const_cast<int64_t*>(topk_idx);  // read only
  a.gw = grad_weights;
  a.glogits = grad_logits;
  return ep::launch_route_backward(a, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

int ep_combine_backward(const ep_problem_t* p, const ep_layout_t* L, const float* topk_weights,
                        const void* grad_out, const void* y, int64_t y_rows, void* grad_y,
                        float* grad_weights, hipStream_t stream) {
  const int rc = check_problem(p);
  if (rc != EP_OK) return rc;
  if (!L || !L->status || y_rows < 0) return EP_EINVAL;
  if (p->num_tokens == 0) return EP_OK;
  if (!L->slot || !topk_weights || !grad_out || !grad_weights) return EP_EINVAL;
  if (y_rows > 0 && (!y || !grad_y)) return EP_EINVAL;
  if (!aligned(grad_out, 2) || !aligned(y, 2) || !aligned(grad_y, 2) || !aligned(topk_weights, 4) ||
      !aligned(grad_weights, 4))
    return EP_EINVAL;
  const int64_t row_bytes = static_cast<int64_t>(p->hidden) * 2, weights = 4 * p->num_tokens * p->topk;
  if (clash({{grad_y, y_rows * row_bytes}, {grad_weights, weights}},
            {{y, y_rows * row_bytes}, {grad_out, p->num_tokens * row_bytes}, {topk_weights, weights}}))
    return EP_EINVAL;
  ep::CombineBackwardArgs a;
  a.go = grad_out;
  a.y = y;
  a.gy = grad_y;
  a.w = topk_weights;
  a.gw = grad_weights;
  a.slot = L->slot;
  a.status = L->status;
  a.generation = L->generation;
  a.T = p->num_tokens;
  a.y_rows = y_rows;
  a.K = p->topk;
  a.H = p->hidden;
  int ve = 8;  // widest vector that divides the row and the bases
  while (ve > 1 && (p->hidden % ve != 0 || !aligned(grad_out, 2 * ve) || !aligned(y, 2 * ve) ||
                    !aligned(grad_y, 2 * ve)))
    ve >>= 1;
  return ep::launch_combine_backward(a, ve, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

size_t ep_lora_workspace_bytes(const ep_problem_t* p, const ep_lora_weights_t* w, int32_t backward) {
  if (check_lora(p, w) != EP_OK) return 0;
  const ep::LoraGeom g = geom_of(p, w, backward != 0);
  return g.bytes() > 0 ? g.bytes() : 16;  // T = 0 needs none; 0 means refused
}

int ep_lora(const ep_problem_t* p, const ep_layout_t* L, const ep_lora_weights_t* w, const void* x,
            int64_t x_row_stride, const void* base, int64_t base_row_stride, void* out,
            int64_t out_row_stride, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_lora(p, w);
  if (rc != EP_OK) return rc;
  if (p->num_tokens == 0) return EP_OK;
  ep::LoraArgs a = {};
  if ((rc = lora_args(p, L, w, &a)) != EP_OK) return rc;
  if ((rc = check_rows(x, x_row_stride, a.H, &a.ldx)) != EP_OK) return rc;
  if ((rc = check_rows(out, out_row_stride, a.N, &a.ldout)) != EP_OK) return rc;
  if (base && (rc = check_rows(base, base_row_stride, a.N, &a.ldbase)) != EP_OK) return rc;
  const ep::LoraGeom g = geom_of(p, w, false);
  const int64_t xrows = a.xmap ? a.T : g.rows, orows = a.omap ? a.T : g.rows;
  const Rows ro = {out, orows, 2LL * a.N, 2 * a.ldout};
  const int64_t na = 2LL * a.E * a.R * a.H, nb = 2LL * a.E * a.R * a.N;
  if (rows_overlap(ro, {x, xrows, 2LL * a.H, 2 * a.ldx}) || rows_overlap(ro, {a.a, 1, na, na}) ||
      rows_overlap(ro, {a.b, 1, nb, nb}))
    return EP_EINVAL;
  if (base && !(base == out && a.ldbase == a.ldout) &&
      rows_overlap(ro, {base, orows, 2LL * a.N, 2 * a.ldbase}))
    return EP_EINVAL;
  if (!workspace || !aligned(workspace, 16)) return EP_EINVAL;
  if (workspace_bytes < g.bytes()) return EP_EWORKSPACE;
  if (workspace_overlaps(workspace, g.bytes(), {ro, {x, xrows, 2LL * a.H, 2 * a.ldx}, {a.a, 1, na, na}, {a.b, 1, nb, nb},
                                                {base, base ? orows : 0, 2LL * a.N, 2 * a.ldbase}}))
    return EP_EINVAL;
  a.x = static_cast<const uint16_t*>(x);
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  set_workspace(&a, g, workspace);
  return ep::launch_lora(a, g, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

int ep_lora_backward(const ep_problem_t* p, const ep_layout_t* L, const ep_lora_weights_t* w,
                     const void* grad_out, int64_t grad_out_row_stride, const void* x,
                     int64_t x_row_stride, const void* grad_base, int64_t grad_base_row_stride,
                     void* grad_x, int64_t grad_x_row_stride, void* grad_a, void* grad_b,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_lora(p, w);
  if (rc != EP_OK) return rc;
  if (!grad_a || !grad_b || !aligned(grad_a, 16) || !aligned(grad_b, 16)) return EP_EINVAL;
  const int64_t na = 2LL * p->num_experts * w->rank * p->hidden, nb = 2LL * p->num_experts * w->rank * w->n_out;
  if (p->num_tokens == 0) {
    // no row: both gradients are zero, by the join kernel
    ep::LoraArgs a = {};
    if ((rc = lora_args(p, L, w, &a)) != EP_OK) return rc;
    a.ga = static_cast<uint16_t*>(grad_a);
    a.gb = static_cast<uint16_t*>(grad_b);
    return ep::launch_lora_backward(a, geom_of(p, w, true), stream) == hipSuccess ? EP_OK : EP_EHIP;
  }
  ep::LoraArgs a = {};
  if ((rc = lora_args(p, L, w, &a)) != EP_OK) return rc;
  if ((rc = check_rows(x, x_row_stride, a.H, &a.ldx)) != EP_OK) return rc;
  if ((rc = check_rows(grad_out, grad_out_row_stride, a.N, &a.ldgo)) != EP_OK) return rc;
  if ((rc = check_rows(grad_x, grad_x_row_stride, a.H, &a.ldout)) != EP_OK) return rc;
  if (grad_base && (rc = check_rows(grad_base, grad_base_row_stride, a.H, &a.ldbase)) != EP_OK) return rc;
  const ep::LoraGeom g = geom_of(p, w, true);
  const int64_t xrows = a.xmap ? a.T : g.rows, orows = a.omap ? a.T : g.rows;
  // no output may overlap an input or another output, but grad_x may be grad_base itself
  const Rows outs[3] = {{grad_x, orows, 2LL * a.H, 2 * a.ldout}, {grad_a, 1, na, na}, {grad_b, 1, nb, nb}};
  const Rows ins[4] = {{x, xrows, 2LL * a.H, 2 * a.ldx},
                       {grad_out, orows, 2LL * a.N, 2 * a.ldgo},
                       {w->a, 1, na, na},
                       {w->b, 1, nb, nb}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j)
      if (rows_overlap(outs[i], ins[j])) return EP_EINVAL;
    for (int j = 0; j < i; ++j)
      if (rows_overlap(outs[i], outs[j])) return EP_EINVAL;
  }
  if (grad_base && !(grad_base == grad_x && a.ldbase == a.ldout)) {
    const Rows rb = {grad_base, orows, 2LL * a.H, 2 * a.ldbase};
    for (int i = 0; i < 3; ++i)
      if (rows_overlap(outs[i], rb)) return EP_EINVAL;
  }
  if (!workspace || !aligned(workspace, 16)) return EP_EINVAL;
  if (workspace_bytes < g.bytes()) return EP_EWORKSPACE;
  if (workspace_overlaps(workspace, g.bytes(), {outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], ins[3],
                                                {grad_base, grad_base ? orows : 0, 2LL * a.H, 2 * a.ldbase}}))
    return EP_EINVAL;
  a.x = static_cast<const uint16_t*>(x);
  a.go = static_cast<const uint16_t*>(grad_out);
  a.base = static_cast<const uint16_t*>(grad_base);
  a.out = static_cast<uint16_t*>(grad_x);
  a.ga = static_cast<uint16_t*>(grad_a);
  a.gb = static_cast<uint16_t*>(grad_b);
  set_workspace(&a, g, workspace);
  return ep::launch_lora_backward(a, g, stream) == hipSuccess ? EP_OK : EP_EHIP;
}

}  // extern "C"
