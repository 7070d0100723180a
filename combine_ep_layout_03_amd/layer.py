"""The operators around dispatch and combine: router, gradients, low-rank
adapters.  A thin binding over the C ABI in include/ep_mi355x_layer.h, in the
manner of the package's other entry points; the formulas stand there.

All tensors of a call must be on one device; the work is enqueued on that
device's current stream.  The gradients are entry points of their own: call
them from a ``torch.autograd.Function`` or a hand-written backward pass.

Single tokens are decoded through these calls, so the host's part counts: the
constant structs of a shape are kept (``functools.lru_cache``), and a tensor
that is as it should be passes its checks in one expression.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import Layout, _dev, _lib, _ptr, _resolve

_BF16, _F32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8
_LOGITS = {_F32: _lib.EP_LOGITS_FP32, _BF16: _lib.EP_LOGITS_BF16}


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape, index: int) -> torch.Tensor:
    """`t` if it is a contiguous tensor of this type and shape (None: any) on
    GPU `index`; raises otherwise."""
    if not (
        isinstance(t, torch.Tensor)
        and t.dtype is dtype
        and t.is_cuda
        and t.is_contiguous()
        and (shape is None or t.shape == shape)
        and t.get_device() == index
    ):
        _dev(t, name, dtype, shape)
        raise ValueError(f"{name} must be on cuda:{index}, as the call's other tensors, got {t.device}")
    return t


def _rows(t: torch.Tensor, name: str, width: int, rows: int, index: int) -> torch.Tensor:
    if (
        isinstance(t, torch.Tensor)
        and t.dtype is _BF16
        and t.is_cuda
        and t.is_contiguous()
        and t.get_device() == index
    ):
        have = t.shape
        if len(have) == 2 and have[1] >= width and have[0] >= rows:
            return t
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be [rows, >= {width}]")
    _check(t, name, _BF16, None, index)
    raise ValueError(f"{name} must be at least [{rows}, {width}], got {tuple(t.shape)}")


def _row_like(t: torch.Tensor | None, rows: int, width: int, other: torch.Tensor) -> torch.Tensor:
    """A new [rows, width] of bf16 on `other`'s GPU; made after `t` where that
    has the shape, which is quicker."""
    if t is not None and t.shape == (rows, width):
        return torch.empty_like(t)
    return other.new_empty((rows, width))


def _call(fn: str, index: int, *args) -> None:
    """The library's `fn` on GPU `index` and its current stream: the library
    launches on the current device."""
    if torch._C._cuda_getDevice() == index:
        rc = getattr(_lib.lib(), fn)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = getattr(_lib.lib(), fn)(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != _lib.EP_OK:
        _lib.check(fn, rc)


def _int32(*values) -> None:
    """Raises for a value that the C structs' int32 fields would cut."""
    for v in values:
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{v} does not fit an int32")


@functools.lru_cache(maxsize=1024)
def _router_struct(*fields):
    _int32(*fields[1:-1])
    return ctypes.byref(_lib.Router(*fields))


@functools.lru_cache(maxsize=1024)
def _problem_struct(*fields):
    _int32(*fields[1:])
    return ctypes.byref(_lib.Problem(*fields))


def _layout_struct(layout: Layout, generation: int) -> _lib.LayoutStruct:
    """The fields of the C struct that these calls read."""
    s = _lib.LayoutStruct()
    s.counts = layout.counts.data_ptr()
    s.offsets = layout.offsets.data_ptr()
    s.slot = layout.slot.data_ptr()
    s.status = layout.status.data_ptr()
    if layout.expert_row_src is not None:
        s.expert_row_src = layout.expert_row_src.data_ptr()
        s.expert_row_capacity = layout.expert_row_capacity
    s.generation = generation
    return s


def _layout_index(layout: Layout, index: int) -> None:
    if layout.slot.get_device() != index:
        raise ValueError(f"layout must be on cuda:{index}, as the call's tensors, got {layout.slot.device}")


def _logits(logits: torch.Tensor):
    """(T, E, EP_LOGITS_*, GPU) of a call's logits."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T, E] tensor")
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    index = logits.get_device() if logits.is_cuda else -1
    _check(logits, "logits", logits.dtype, None, index)
    T, E = logits.shape
    return T, E, kind, index


def ep_route(
    logits: torch.Tensor,
    topk: int,
    score: int = _lib.EP_SCORE_SOFTMAX,
    bias: torch.Tensor | None = None,
    num_groups: int = 0,
    topk_groups: int = 0,
    group_top: int = 1,
    renormalize: bool = False,
    scale: float = 1.0,
    token_mask: torch.Tensor | None = None,
    out: tuple[torch.Tensor, torch.Tensor] | None = None,
) -> tuple[torch.Tensor, torch.Tensor]:
    """Choose each token's ``topk`` experts from logits (fp32 or bf16 [T, E]).

    Returns (topk_idx int64 [T, K], topk_weights fp32 [T, K]), what
    ``ep_layout`` and ``ep_combine`` take.  Experts are chosen by score +
    ``bias`` (fp32 [E]), or by logit without a bias, in descending order, ties
    to the lowest index, compared as in binary64; the weights are the scores
    (EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID) of the chosen, divided by their sum
    with ``renormalize``, times ``scale``.  With ``num_groups`` the choice is
    limited to ``topk_groups`` of the contiguous expert groups, the ones with
    the largest sum of ``group_top`` (1 or 2) best values.  A NaN or -inf
    logit takes an expert out; ``token_mask`` (bool or uint8 [T]) False takes
    a token out; entries without an expert are -1 with weight 0.  ``out`` is
    a pair of tensors to write to."""
    T, E, kind, index = _logits(logits)
    K = int(topk)
    if K < 1:
        raise ValueError("topk must be at least 1")
    r = _router_struct(T, E, K, int(score), kind, int(num_groups), int(topk_groups), int(group_top),
                       int(bool(renormalize)), float(scale))
    if bias is not None:
        _check(bias, "bias", _F32, (E,), index)
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, _U8):
            raise TypeError("token_mask must be bool or uint8")
        _check(token_mask, "token_mask", token_mask.dtype, (T,), index)
    if out is None:
        idx = logits.new_empty((T, K), dtype=_I64)
        w = logits.new_empty((T, K), dtype=_F32)
    else:
        idx, w = out
        _check(idx, "out[0]", _I64, (T, K), index)
        _check(w, "out[1]", _F32, (T, K), index)
    _call("ep_route", index, r, logits.data_ptr(), _ptr(bias), _ptr(token_mask), idx.data_ptr(), w.data_ptr())
    return idx, w


def ep_route_backward(
    grad_weights: torch.Tensor,
    logits: torch.Tensor,
    topk_idx: torch.Tensor,
    score: int = _lib.EP_SCORE_SOFTMAX,
    renormalize: bool = False,
    scale: float = 1.0,
    out: torch.Tensor | None = None,
) -> torch.Tensor:
    """Gradient of ``ep_route``'s weights with respect to the logits, given
    grad_weights (fp32 [T, K], for example ``ep_combine_backward``'s), the
    logits, the choice topk_idx (int64 [T, K]) and the same score,
    renormalize and scale.  Returns [T, E] in the logits' type."""
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, E, kind, index = _logits(logits)
    K = topk_idx.shape[1]
    r = _router_struct(T, E, K, int(score), kind, 0, 0, 1, int(bool(renormalize)), float(scale))
    _check(topk_idx, "topk_idx", _I64, (T, K), index)
    _check(grad_weights, "grad_weights", _F32, (T, K), index)
    if out is None:
        out = torch.empty_like(logits)
    else:
        _check(out, "out", logits.dtype, (T, E), index)
    _call("ep_route_backward", index, r, logits.data_ptr(), topk_idx.data_ptr(), grad_weights.data_ptr(),
          out.data_ptr())
    return out


def ep_combine_backward(
    grad_out: torch.Tensor,
    y: torch.Tensor,
    layout: Layout,
    topk_weights: torch.Tensor,
    grad_y: torch.Tensor | None = None,
    grad_weights: torch.Tensor | None = None,
) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``ep_combine`` (either order): from grad_out (bf16 [T, H]),
    the expert-output rows y (bf16 [rows, H]) and the weights (fp32 [T, K]),
    returns (grad_y bf16 [rows, H], grad_weights fp32 [T, K]).  Rows of grad_y
    that no selection owns are left as they were (undefined if grad_y is
    allocated here).  A bias row's gradient is grad_out itself.  ``layout``
    may be a LayoutHandle."""
    layout, gen = _resolve(layout)
    if not isinstance(y, torch.Tensor) or y.dim() != 2:
        raise ValueError("y must be [rows, H]")
    index = y.get_device() if y.is_cuda else -1
    _check(y, "y", _BF16, None, index)
    T, K = layout.num_tokens, layout.topk
    rows, H = y.shape
    _check(grad_out, "grad_out", _BF16, (T, H), index)
    _check(topk_weights, "topk_weights", _F32, (T, K), index)
    if grad_y is None:
        grad_y = torch.empty_like(y)
    else:
        _check(grad_y, "grad_y", _BF16, (rows, H), index)
    if grad_weights is None:
        grad_weights = torch.empty_like(topk_weights)
    else:
        _check(grad_weights, "grad_weights", _F32, (T, K), index)
    _layout_index(layout, index)
    p = _problem_struct(T, H, K, layout.num_experts, layout.num_groups, layout.expert_alignment, 0)
    s = _layout_struct(layout, gen)
    _call("ep_combine_backward", index, p, ctypes.byref(s), topk_weights.data_ptr(), grad_out.data_ptr(),
          y.data_ptr(), rows, grad_y.data_ptr(), grad_weights.data_ptr())
    return grad_y, grad_weights


@functools.lru_cache(maxsize=1024)
def _lora_workspace(T, H, K, E, G, A, flags, R, N, wflags, backward) -> int:
    _int32(R, N)
    w = _lib.LoraWeights(None, None, None, R, N, wflags)
    return int(_lib.lib().ep_lora_workspace_bytes(_problem_struct(T, H, K, E, G, A, flags), ctypes.byref(w),
                                                  backward))


def ep_lora_workspace_bytes(layout: Layout, hidden: int, n_out: int, rank: int, backward: bool = False) -> int:
    """Bytes of workspace ``ep_lora`` (or ``ep_lora_backward``) needs on this
    layout; 0 if it would refuse the sizes.  The backward pass's holds partial
    gradients and grows with the rows above 131,072 (the C header has the rule)."""
    layout, _ = _resolve(layout)
    return _lora_workspace(layout.num_tokens, int(hidden), layout.topk, layout.num_experts, layout.num_groups,
                           layout.expert_alignment, 0, int(rank), int(n_out), 0, int(backward))


def _lora_args(layout, gen, a, b, scales, gather, scatter, backward, workspace):
    """Checks of a call's adapters, row modes and workspace, and its structs:
    (R, N, H, rows of x, rows of out, GPU, problem, layout, adapters, workspace)."""
    for t in (a, b):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError("a must be [E, R, H] and b [E, N, R]")
    index = a.get_device() if a.is_cuda else -1
    _check(a, "a", _BF16, None, index)
    E, R, H = a.shape
    N = b.shape[1]
    if E != layout.num_experts:
        raise ValueError("a must hold one [R, H] matrix per expert of the layout")
    _check(b, "b", _BF16, (E, N, R), index)
    if scales is not None:
        _check(scales, "scales", _F32, (E,), index)
    _layout_index(layout, index)
    rows, T = layout.max_expert_rows(), layout.num_tokens
    if (gather or scatter) and (layout.expert_row_src is None or layout.expert_row_capacity < rows):
        raise ValueError("gather and scatter need a layout computed with expert_row_src=True")
    if scatter and layout.topk != 1:
        raise ValueError("scatter needs a layout with one selection per token")
    wflags = _lib.EP_LORA_SCATTER_ROWS if scatter else 0
    shape = (T, H, layout.topk, E, layout.num_groups, layout.expert_alignment,
             _lib.EP_FLAG_GATHER_ROWS if gather else 0)
    if workspace is None:
        workspace = a.new_empty(_lora_workspace(*shape, R, N, wflags, backward), dtype=_U8)
    else:
        _check(workspace, "workspace", _U8, None, index)
    w = _lib.LoraWeights(a.data_ptr(), b.data_ptr(), _ptr(scales), R, N, wflags)
    return (R, N, H, T if gather else rows, T if scatter else rows, index, _problem_struct(*shape),
            ctypes.byref(_layout_struct(layout, gen)), ctypes.byref(w), workspace)


def ep_lora(
    x: torch.Tensor,
    layout: Layout,
    a: torch.Tensor,
    b: torch.Tensor,
    base: torch.Tensor | None = None,
    scales: torch.Tensor | None = None,
    gather: bool = False,
    scatter: bool = False,
    out: torch.Tensor | None = None,
    workspace: torch.Tensor | None = None,
) -> torch.Tensor:
    """Low-rank adapters beside a projection: out = base + scales[e] * (x
    a[e]^T) b[e]^T for the rows of each expert e of the layout.

    a: bf16 [E, R, H], b: bf16 [E, N, R] (R a multiple of 8 up to 128, H and N
    multiples of 8), scales: fp32 [E] or None (1).  x (bf16) holds receive rows,
    or with ``gather`` the token rows, as in ``ep_expert_gemm``; base and out
    (bf16) hold receive rows, or with ``scatter`` token rows (one selection
    per token).  For requests with adapters of their own, the layout is
    ``ep_layout(adapter_ids[:, None], E, expert_row_src=True)`` with id -1 for
    none, and both flags are set.  ``out`` may be ``base`` (the delta is added
    in place); with ``scatter`` the token rows without an adapter become
    base's (zeros without one), other rows of no selection are not written.
    ``workspace`` (uint8, ``ep_lora_workspace_bytes``) is allocated if not
    given; calls that may overlap need their own."""
    layout, gen = _resolve(layout)
    R, N, H, xrows, orows, index, p, s, w, workspace = _lora_args(layout, gen, a, b, scales, gather, scatter, 0,
                                                                  workspace)
    _rows(x, "x", H, xrows, index)
    if base is not None:
        _rows(base, "base", N, orows, index)
    if out is None:
        out = _row_like(base, orows, N, x)
    else:
        _rows(out, "out", N, orows, index)
    _call("ep_lora", index, p, s, w, x.data_ptr(), x.shape[1], _ptr(base), 0 if base is None else base.shape[1],
          out.data_ptr(), out.shape[1], workspace.data_ptr(), workspace.numel())
    return out


def ep_lora_backward(
    grad_out: torch.Tensor,
    x: torch.Tensor,
    layout: Layout,
    a: torch.Tensor,
    b: torch.Tensor,
    scales: torch.Tensor | None = None,
    gather: bool = False,
    scatter: bool = False,
    grad_base: torch.Tensor | None = None,
    grad_x: torch.Tensor | None = None,
    grad_a: torch.Tensor | None = None,
    grad_b: torch.Tensor | None = None,
    workspace: torch.Tensor | None = None,
) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ``ep_lora``: (grad_x, grad_a, grad_b), all bf16, from
    grad_out (rows as out's) and the forward call's x, layout, adapters, scales
    and row modes.

    grad_x has out's rows (H wide): with ``gather`` and several selections per
    token each receive row keeps its own, and ``ep_combine`` with unit weights
    adds them up.  ``grad_base`` (same rows) is added to it: the gradient that
    the projection beside the adapter sends to x; it may be ``grad_x``.  Rows
    of no selection are treated as ``ep_lora`` treats out's.  An expert
    without rows gets zero gradients.  The gradient of base is grad_out
    itself."""
    layout, gen = _resolve(layout)
    R, N, H, xrows, orows, index, p, s, w, workspace = _lora_args(layout, gen, a, b, scales, gather, scatter, 1,
                                                                  workspace)
    _rows(x, "x", H, xrows, index)
    _rows(grad_out, "grad_out", N, orows, index)
    if grad_base is not None:
        _rows(grad_base, "grad_base", H, orows, index)
    if grad_x is None:
        grad_x = _row_like(x, orows, H, x)
    else:
        _rows(grad_x, "grad_x", H, orows, index)
    if grad_a is None:
        grad_a = torch.empty_like(a)
    else:
        _check(grad_a, "grad_a", _BF16, a.shape, index)
    if grad_b is None:
        grad_b = torch.empty_like(b)
    else:
        _check(grad_b, "grad_b", _BF16, b.shape, index)
    _call("ep_lora_backward", index, p, s, w, grad_out.data_ptr(), grad_out.shape[1], x.data_ptr(), x.shape[1],
          _ptr(grad_base), 0 if grad_base is None else grad_base.shape[1], grad_x.data_ptr(), grad_x.shape[1],
          grad_a.data_ptr(), grad_b.data_ptr(), workspace.data_ptr(), workspace.numel())
    return grad_x, grad_a, grad_b
