// Argument checks shared by the C-ABI entry points of the layer operators.
#pragma once

#include <limits.h>
#include <stdint.h>

#include <initializer_list>

#include "ep_mi355x.h"

namespace ep {
namespace checks {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Do [a, a + na) and [b, b + nb) share a byte?
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}

struct Span {
  const void* p;  // null: not there
  int64_t n;      // bytes
};
// Does an output share a byte with an input or another output?
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* other = outs.begin(); other != o; ++other)
      if (overlap(o->p, o->n, other->p, other->n)) return true;
    for (const Span& i : ins)
      if (overlap(o->p, o->n, i.p, i.n)) return true;
  }
  return false;
}

// The shape checks of ep_mi355x.h's calls, for the fields a call on a
// finished layout uses.
inline int check_problem(const ep_problem_t* p) {
  if (!p) return EP_EINVAL;
  if (p->num_tokens < 0 || p->hidden < 1 || p->topk < 1 || p->num_experts < 1 || p->num_groups < 0)
    return EP_EINVAL;
  if (p->expert_alignment < 0 || p->expert_alignment > (1 << 20)) return EP_EINVAL;
  if (p->flags & ~(EP_FLAG_ZERO_PADDING | EP_FLAG_GATHER_ROWS | EP_FLAG_PACKED_WEIGHTS)) return EP_EINVAL;
  if (p->topk > EP_MAX_TOPK || static_cast<int64_t>(p->num_experts) + p->num_groups > EP_MAX_KEYS)
    return EP_ENOTSUP;
  const int64_t pad = static_cast<int64_t>(p->num_experts) *
                      (p->expert_alignment > 1 ? p->expert_alignment - 1 : 0);
  if (p->num_tokens > (static_cast<int64_t>(INT32_MAX) - pad) / p->topk) return EP_ENOTSUP;
  return EP_OK;
}

// Do two sets of rows (bytes: width each, pitch ld apart) share a byte?  Rows
// of one pitch whose columns are apart (two parts of one buffer) do not.
struct Rows {
  const void* p;
  int64_t n, width, ld;
};
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (a.n == 0 || b.n == 0 || !overlap(a.p, (a.n - 1) * a.ld + a.width, b.p, (b.n - 1) * b.ld + b.width))
    return false;
  if (a.ld != b.ld) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const int64_t ld = a.ld;
  const int64_t d = pb >= pa ? static_cast<int64_t>((pb - pa) % static_cast<uintptr_t>(ld))
                             : (ld - static_cast<int64_t>((pa - pb) % static_cast<uintptr_t>(ld))) % ld;
  return !(d >= a.width && d + b.width <= ld);
}

inline bool workspace_overlaps(const void* workspace, size_t bytes, std::initializer_list<Rows> used) {
  for (const Rows& r : used)
    if (r.n > 0 && overlap(workspace, static_cast<int64_t>(bytes), r.p, (r.n - 1) * r.ld + r.width)) return true;
  return false;
}

// Rows of the receive buffers at most, the padding of aligned segments included.
inline int64_t max_rows(const ep_problem_t* p) {
  const int64_t pad = static_cast<int64_t>(p->num_experts) *
                      (p->expert_alignment > 1 ? p->expert_alignment - 1 : 0);
  return p->num_tokens * p->topk + pad;
}

// Rows of a selection at most: what the experts' counts add up to.
inline int64_t selections(const ep_problem_t* p) { return p->num_tokens * p->topk; }

// A matrix of rows: stride (0 = width), alignment.
inline int check_rows(const void* p, int64_t stride, int32_t width, int64_t* ld) {
  *ld = stride == 0 ? width : stride;
  return p && aligned(p, 16) && *ld >= width && *ld % 8 == 0 ? EP_OK : EP_EINVAL;
}

}  // namespace checks
}  // namespace ep
