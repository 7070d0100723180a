"""The operators around dispatch and combine: router, gradients, low-rank
adapters.  A thin binding over the C ABI in include/ep_mi355x_layer.h, in the
manner of the package's other entry points; the formulas stand there.

All tensors of a call must be on one device; the work is enqueued on that
device's current stream.  The gradients are entry points of their own: call
them from a ``torch.autograd.Function`` or a hand-written backward pass.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import Layout, _dev, _lib, _problem, _ptr, _resolve, _stream

_HERE = contextlib.nullcontext()
_LOGITS = {torch.float32: _lib.EP_LOGITS_FP32, torch.bfloat16: _lib.EP_LOGITS_BF16}


def _on_device(device: torch.device, *others: torch.Tensor | None):
    """Run on `device`: the library launches on the current device."""
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"all tensors must be on {device}, got one on {t.device}")
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _router(logits, topk, score, renormalize, scale, num_groups=0, topk_groups=0, group_top=1) -> _lib.Router:
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T, E] tensor")
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    _dev(logits, "logits", logits.dtype)
    T, E = logits.shape
    return _lib.Router(T, E, int(topk), int(score), _LOGITS[logits.dtype], int(num_groups), int(topk_groups),
                       int(group_top), int(bool(renormalize)), float(scale))


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
    r = _router(logits, topk, score, renormalize, scale, num_groups, topk_groups, group_top)
    T, E, K = logits.shape[0], logits.shape[1], int(topk)
    if bias is not None:
        _dev(bias, "bias", torch.float32, (E,))
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("token_mask must be bool or uint8")
        _dev(token_mask, "token_mask", token_mask.dtype, (T,))
    if K < 1:
        raise ValueError("topk must be at least 1")
    if out is None:
        idx = torch.empty(T, K, dtype=torch.int64, device=logits.device)
        w = torch.empty(T, K, dtype=torch.float32, device=logits.device)
    else:
        idx, w = out
        _dev(idx, "out[0]", torch.int64, (T, K))
        _dev(w, "out[1]", torch.float32, (T, K))
    with _on_device(logits.device, bias, token_mask, idx, w):
        rc = _lib.lib().ep_route(ctypes.byref(r), _ptr(logits), _ptr(bias), _ptr(token_mask), _ptr(idx), _ptr(w),
                                 _stream(logits.device))
    _lib.check("ep_route", rc)
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
    K = topk_idx.shape[1]
    r = _router(logits, K, score, renormalize, scale)
    T = logits.shape[0]
    _dev(topk_idx, "topk_idx", torch.int64, (T, K))
    _dev(grad_weights, "grad_weights", torch.float32, (T, K))
    if out is None:
        out = torch.empty_like(logits)
    else:
        _dev(out, "out", logits.dtype, logits.shape)
    with _on_device(logits.device, topk_idx, grad_weights, out):
        rc = _lib.lib().ep_route_backward(ctypes.byref(r), _ptr(logits), _ptr(topk_idx), _ptr(grad_weights),
                                          _ptr(out), _stream(logits.device))
    _lib.check("ep_route_backward", rc)
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
    _dev(y, "y", torch.bfloat16)
    T, K, H = layout.num_tokens, layout.topk, y.shape[1]
    _dev(grad_out, "grad_out", torch.bfloat16, (T, H))
    _dev(topk_weights, "topk_weights", torch.float32, (T, K))
    if grad_y is None:
        grad_y = torch.empty_like(y)
    else:
        _dev(grad_y, "grad_y", torch.bfloat16, y.shape)
    if grad_weights is None:
        grad_weights = torch.empty(T, K, dtype=torch.float32, device=y.device)
    else:
        _dev(grad_weights, "grad_weights", torch.float32, (T, K))
    p = _problem(T, H, K, layout.num_experts, layout.num_groups, layout.expert_alignment)
    s = layout.struct(gen)
    with _on_device(y.device, grad_out, topk_weights, grad_y, grad_weights, layout.slot):
        rc = _lib.lib().ep_combine_backward(ctypes.byref(p), ctypes.byref(s), _ptr(topk_weights), _ptr(grad_out),
                                            _ptr(y), int(y.shape[0]), _ptr(grad_y), _ptr(grad_weights),
                                            _stream(y.device))
    _lib.check("ep_combine_backward", rc)
    return grad_y, grad_weights


@functools.lru_cache(maxsize=256)
def _lora_workspace(T, H, K, E, G, A, flags, R, N, wflags, backward) -> int:
    p = _problem(T, H, K, E, G, A, flags)
    w = _lib.LoraWeights(None, None, None, R, N, wflags)
    return int(_lib.lib().ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), backward))


def ep_lora_workspace_bytes(layout: Layout, hidden: int, n_out: int, rank: int, backward: bool = False) -> int:
    """Bytes of workspace ``ep_lora`` (or ``ep_lora_backward``) needs on this
    layout; 0 if it would refuse the sizes."""
    layout, _ = _resolve(layout)
    return _lora_workspace(layout.num_tokens, int(hidden), layout.topk, layout.num_experts, layout.num_groups,
                           layout.expert_alignment, 0, int(rank), int(n_out), 0, int(backward))


def _rows(t, name, width, rows):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be [rows, >= {width}]")
    _dev(t, name, torch.bfloat16)
    if t.shape[1] < width or t.shape[0] < rows:
        raise ValueError(f"{name} must be at least [{rows}, {width}], got {tuple(t.shape)}")
    return t


def _adapters(layout, a, b, scales, gather, scatter):
    """Checks of a call's adapters and row modes; (E, R, N, H, rows of x, rows of out)."""
    for name, t in (("a", a), ("b", b)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError("a must be [E, R, H] and b [E, N, R]")
        _dev(t, name, torch.bfloat16)
    E, R, H = a.shape
    N = b.shape[1]
    if E != layout.num_experts:
        raise ValueError("a must hold one [R, H] matrix per expert of the layout")
    _dev(b, "b", torch.bfloat16, (E, N, R))
    if scales is not None:
        _dev(scales, "scales", torch.float32, (E,))
    rows = layout.max_expert_rows()
    if (gather or scatter) and (layout.expert_row_src is None or layout.expert_row_capacity < rows):
        raise ValueError("gather and scatter need a layout computed with expert_row_src=True")
    if scatter and layout.topk != 1:
        raise ValueError("scatter needs a layout with one selection per token")
    T = layout.num_tokens
    return E, R, N, H, T if gather else rows, T if scatter else rows


def _lora_structs(layout, gen, a, b, scales, R, N, H, gather, scatter, backward, workspace):
    flags = _lib.EP_FLAG_GATHER_ROWS if gather else 0
    wflags = _lib.EP_LORA_SCATTER_ROWS if scatter else 0
    shape = (layout.num_tokens, H, layout.topk, layout.num_experts, layout.num_groups, layout.expert_alignment)
    p = _problem(*shape, flags)
    w = _lib.LoraWeights(_ptr(a), _ptr(b), _ptr(scales), R, N, wflags)
    need = _lora_workspace(*shape, flags, R, N, wflags, int(backward))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
    else:
        _dev(workspace, "workspace", torch.uint8)
    return p, layout.struct(gen), w, workspace


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
    E, R, N, H, xrows, orows = _adapters(layout, a, b, scales, gather, scatter)
    _rows(x, "x", H, xrows)
    if base is not None:
        _rows(base, "base", N, orows)
    if out is None:
        out = torch.empty(orows, N, dtype=torch.bfloat16, device=x.device)
    else:
        _rows(out, "out", N, orows)
    with _on_device(x.device, a, b, base, scales, out, workspace, layout.slot):
        p, s, w, workspace = _lora_structs(layout, gen, a, b, scales, R, N, H, gather, scatter, False, workspace)
        rc = _lib.lib().ep_lora(
            ctypes.byref(p), ctypes.byref(s), ctypes.byref(w), _ptr(x), x.shape[1], _ptr(base),
            0 if base is None else base.shape[1], _ptr(out), out.shape[1], _ptr(workspace), workspace.numel(),
            _stream(x.device),
        )
    _lib.check("ep_lora", rc)
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
    E, R, N, H, xrows, orows = _adapters(layout, a, b, scales, gather, scatter)
    _rows(x, "x", H, xrows)
    _rows(grad_out, "grad_out", N, orows)
    if grad_base is not None:
        _rows(grad_base, "grad_base", H, orows)
    if grad_x is None:
        grad_x = torch.empty(orows, H, dtype=torch.bfloat16, device=x.device)
    else:
        _rows(grad_x, "grad_x", H, orows)
    if grad_a is None:
        grad_a = torch.empty_like(a)
    else:
        _dev(grad_a, "grad_a", torch.bfloat16, a.shape)
    if grad_b is None:
        grad_b = torch.empty_like(b)
    else:
        _dev(grad_b, "grad_b", torch.bfloat16, b.shape)
    with _on_device(x.device, a, b, scales, grad_out, grad_base, grad_x, grad_a, grad_b, workspace, layout.slot):
        p, s, w, workspace = _lora_structs(layout, gen, a, b, scales, R, N, H, gather, scatter, True, workspace)
        rc = _lib.lib().ep_lora_backward(
            ctypes.byref(p), ctypes.byref(s), ctypes.byref(w), _ptr(grad_out), grad_out.shape[1], _ptr(x),
            x.shape[1], _ptr(grad_base), 0 if grad_base is None else grad_base.shape[1], _ptr(grad_x),
            grad_x.shape[1], _ptr(grad_a), _ptr(grad_b), _ptr(workspace), workspace.numel(), _stream(x.device),
        )
    _lib.check("ep_lora_backward", rc)
    return grad_x, grad_a, grad_b
