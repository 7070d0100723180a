"""The experts' layers and the router's balance loss: products with bias,
activation and residual in their epilogue, per-expert counts, and their
gradients.  A thin binding over the C ABI in include/ep_mi355x_expert.h, in
the manner of the package's other entry points; the formulas stand there.

All tensors of a call must be on one device; the work is enqueued on that
device's current stream.  The gradients are entry points of their own: call
them from a ``torch.autograd.Function`` or a hand-written backward pass.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import Layout, _lib, _ptr, _resolve
from .layer import _BF16, _F32, _I64, _LOGITS, _U8, _call, _check, _int32, _layout_index, _layout_struct, _logits, \
    _problem_struct, _row_like, _rows

_I32 = torch.int32


@functools.lru_cache(maxsize=1024)
def _linear_workspace(T, H, K, E, G, A, flags, N, activation, gated) -> int:
    _int32(N, activation)
    lin = _lib.Linear(None, None, N, activation, gated)
    return int(_lib.lib().ep_expert_linear_workspace_bytes(_problem_struct(T, H, K, E, G, A, flags),
                                                           ctypes.byref(lin)))


def ep_expert_linear_workspace_bytes(layout: Layout, hidden: int, n_out: int, gated: bool = False) -> int:
    """Bytes of workspace ``ep_expert_linear_backward`` needs on this layout; 0
    if it would refuse the sizes."""
    layout, _ = _resolve(layout)
    return _linear_workspace(layout.num_tokens, int(hidden), layout.topk, layout.num_experts, layout.num_groups,
                             layout.expert_alignment, 0, int(n_out), 0, int(bool(gated)))


def _linear_args(layout, gen, w, bias, activation, gated, gather):
    """Checks of a call's weights and row mode, and its structs: (W, N, H,
    receive rows, rows of x, GPU, shape, problem, layout, linear)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be [E, N, H], or [E, 2 N, H] with gated")
    index = w.get_device() if w.is_cuda else -1
    _check(w, "w", _BF16, None, index)
    E, W, H = w.shape
    gated = int(bool(gated))
    if gated and W % 2:
        raise ValueError("with gated, w must hold as many gate rows as others")
    if E != layout.num_experts:
        raise ValueError("w must hold one matrix per expert of the layout")
    N = W // 2 if gated else W
    if bias is not None:
        _check(bias, "bias", _BF16, (E, W), index)
    _layout_index(layout, index)
    rows = layout.max_expert_rows()
    if gather and (layout.expert_row_src is None or layout.expert_row_capacity < rows):
        raise ValueError("gather needs a layout computed with expert_row_src=True")
    shape = (layout.num_tokens, H, layout.topk, E, layout.num_groups, layout.expert_alignment,
             _lib.EP_FLAG_GATHER_ROWS if gather else 0)
    _int32(N, int(activation))
    lin = _lib.Linear(w.data_ptr(), _ptr(bias), N, int(activation), gated)
    return (W, N, H, rows, layout.num_tokens if gather else rows, index, shape, _problem_struct(*shape),
            ctypes.byref(_layout_struct(layout, gen)), ctypes.byref(lin))


def _stride(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.shape[1]


def ep_expert_linear(
    x: torch.Tensor,
    layout: Layout,
    w: torch.Tensor,
    bias: torch.Tensor | None = None,
    activation: int = _lib.EP_ACT_NONE,
    gated: bool = False,
    residual: torch.Tensor | None = None,
    gather: bool = False,
    out: torch.Tensor | None = None,
    pre: torch.Tensor | None = None,
) -> torch.Tensor:
    """An expert's layer over the layout's segments: z = x w[e]^T + bias[e], out
    = activation(z) + residual for the rows of each expert e, or with ``gated``
    (w holds N gate rows, then N more) activation(z[:, :N]) * z[:, N:] +
    residual.

    w: bf16 [E, N, H] ([E, 2 N, H] with ``gated``), bias: bf16 [E, N] ([E, 2
    N]), H and N multiples of 8; activation: EP_ACT_NONE, _RELU, _SILU, _GELU
    or _GELU_TANH.  x (bf16) holds receive rows, or with ``gather`` the token
    rows, as in ``ep_expert_gemm``; residual and out (bf16, at least N wide)
    hold receive rows, and out may be residual itself.  ``pre`` (bf16 rows, at
    least w.shape[1] wide) gets z, which ``ep_expert_linear_backward`` takes.
    Rows of no selection are not written."""
    layout, gen = _resolve(layout)
    W, N, H, rows, xrows, index, _, p, s, lin = _linear_args(layout, gen, w, bias, activation, gated, gather)
    _rows(x, "x", H, xrows, index)
    if residual is not None:
        _rows(residual, "residual", N, rows, index)
    if pre is not None:
        _rows(pre, "pre", W, rows, index)
    if out is None:
        out = _row_like(residual, rows, N, x)
    else:
        _rows(out, "out", N, rows, index)
    _call("ep_expert_linear", index, p, s, lin, x.data_ptr(), x.shape[1], _ptr(residual), _stride(residual),
          out.data_ptr(), out.shape[1], _ptr(pre), _stride(pre))
    return out


def ep_expert_linear_backward(
    grad_out: torch.Tensor,
    x: torch.Tensor,
    layout: Layout,
    w: torch.Tensor,
    pre: torch.Tensor | None = None,
    activation: int = _lib.EP_ACT_NONE,
    gated: bool = False,
    gather: bool = False,
    bias: bool = False,
    grad_x: torch.Tensor | None = None,
    grad_w: torch.Tensor | None = None,
    grad_bias: torch.Tensor | None = None,
    grad_pre: torch.Tensor | None = None,
    workspace: torch.Tensor | None = None,
    needs: tuple[bool, bool] = (True, True),
) -> tuple[torch.Tensor | None, torch.Tensor | None, torch.Tensor | None, torch.Tensor | None]:
    """Gradients of ``ep_expert_linear``: (grad_x, grad_w, grad_bias, grad_pre),
    all bf16, from grad_out (rows as out's) and the forward call's x, layout,
    weights, activation and row mode, and ``pre`` as it wrote it.

    grad_pre is the gradient of the values before the activation; without
    activation and gate it is grad_out itself (None is returned, and pre is not
    taken).  It may be written over ``pre``.  grad_x holds receive rows; with
    ``gather`` each keeps its own, and ``ep_combine`` with unit weights adds a
    token's.  grad_bias is computed if ``bias`` is set or the tensor is given.
    ``needs`` says whether grad_x and grad_w are wanted (None for one that is
    not; the bias's comes with the weights').  An expert without rows gets zero
    weight gradients; rows of no selection are not written.  The gradient of
    the residual is grad_out itself.  ``workspace`` (uint8,
    ``ep_expert_linear_workspace_bytes``) is for the weights' and allocated if
    not given; calls that may overlap need their own."""
    layout, gen = _resolve(layout)
    W, N, H, rows, xrows, index, shape, p, s, lin = _linear_args(layout, gen, w, None, activation, gated, gather)
    _rows(grad_out, "grad_out", N, rows, index)
    need_x, need_w = needs
    bias = bias or grad_bias is not None
    if bias and not need_w:
        raise ValueError("grad_bias comes with grad_w")
    if (grad_x is not None and not need_x) or (grad_w is not None and not need_w):
        raise ValueError("a gradient that needs leaves out was given a tensor")
    if need_w:
        _rows(x, "x", H, xrows, index)
    if int(activation) == _lib.EP_ACT_NONE and not gated:
        if pre is not None or grad_pre is not None:
            raise ValueError("without activation and gate, pre and grad_pre are not taken")
    else:
        if pre is None:
            raise ValueError("the gradient of an activation or gate needs pre")
        _rows(pre, "pre", W, rows, index)
        if grad_pre is None:
            grad_pre = _row_like(pre, rows, W, pre)
        else:
            _rows(grad_pre, "grad_pre", W, rows, index)
    if need_x:
        if grad_x is None:
            grad_x = _row_like(x, rows, H, grad_out)
        else:
            _rows(grad_x, "grad_x", H, rows, index)
    if need_w:
        if grad_w is None:
            grad_w = torch.empty_like(w)
        else:
            _check(grad_w, "grad_w", _BF16, w.shape, index)
    if bias:
        if grad_bias is None:
            grad_bias = w.new_empty((w.shape[0], W))
        else:
            _check(grad_bias, "grad_bias", _BF16, (w.shape[0], W), index)
    if workspace is not None:
        _check(workspace, "workspace", _U8, None, index)
    elif need_w:
        workspace = w.new_empty(_linear_workspace(*shape, N, int(activation), int(bool(gated))), dtype=_U8)
    _call("ep_expert_linear_backward", index, p, s, lin, grad_out.data_ptr(), grad_out.shape[1],
          x.data_ptr() if need_w else None, x.shape[1] if need_w else 0, _ptr(pre), _stride(pre), _ptr(grad_pre),
          _stride(grad_pre), _ptr(grad_x), _stride(grad_x), _ptr(grad_w), _ptr(grad_bias), _ptr(workspace),
          0 if workspace is None else workspace.numel())
    return grad_x, grad_w, grad_bias, grad_pre


@functools.lru_cache(maxsize=1024)
def _balance_struct(*fields):
    _int32(*fields[1:-1])
    return ctypes.byref(_lib.Balance(*fields))


@functools.lru_cache(maxsize=1024)
def _balance_workspace(*fields) -> int:
    return int(_lib.lib().ep_balance_workspace_bytes(_balance_struct(*fields)))


def ep_balance_workspace_bytes(num_tokens: int, num_experts: int, topk: int, num_seqs: int = 1) -> int:
    """Bytes of workspace ``ep_balance_loss`` needs; 0 if it would refuse the
    sizes."""
    return _balance_workspace(int(num_tokens), int(num_experts), int(topk), 0, 0, int(num_seqs), 1.0)


def _balance_args(logits, topk, score, coef, seq_offsets, token_mask):
    T, E, kind, index = _logits(logits)
    B = 1
    if seq_offsets is not None:
        if not isinstance(seq_offsets, torch.Tensor) or seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
            raise ValueError("seq_offsets must be [B + 1]")
        B = seq_offsets.numel() - 1
        _check(seq_offsets, "seq_offsets", _I32, None, index)
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, _U8):
            raise TypeError("token_mask must be bool or uint8")
        _check(token_mask, "token_mask", token_mask.dtype, (T,), index)
    return T, E, B, index, (T, E, int(topk), int(score), kind, B, float(coef))


def ep_balance_loss(
    logits: torch.Tensor,
    topk_idx: torch.Tensor,
    score: int = _lib.EP_SCORE_SOFTMAX,
    coef: float = 1.0,
    seq_offsets: torch.Tensor | None = None,
    token_mask: torch.Tensor | None = None,
    workspace: torch.Tensor | None = None,
) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """The balance loss of a router's choice topk_idx (int64 [T, K]) by its
    logits (fp32 or bf16 [T, E]), sequence by sequence: coef times the mean over
    the sequences of E / (K n) sum_e counts[e] mean[e], n a sequence's tokens
    and mean[e] their mean score of expert e, each token's scores over their
    sum.

    Returns (loss fp32 [1], counts int32 [B, E], tokens int32 [B], mean fp32
    [B, E]).  Sequence b is the tokens [seq_offsets[b], seq_offsets[b + 1]) of
    an int32 [B + 1], ascending, or all T without; tokens outside of every
    sequence, and those whose ``token_mask`` (bool or uint8 [T]) is False, have
    no part.  ``workspace`` (uint8, ``ep_balance_workspace_bytes``) is allocated
    if not given; calls that may overlap need their own."""
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    K = topk_idx.shape[1]
    T, E, B, index, fields = _balance_args(logits, K, score, coef, seq_offsets, token_mask)
    _check(topk_idx, "topk_idx", _I64, (T, K), index)
    if workspace is None:
        workspace = logits.new_empty(_balance_workspace(*fields), dtype=_U8)
    else:
        _check(workspace, "workspace", _U8, None, index)
    loss = logits.new_empty(1, dtype=_F32)
    counts = logits.new_empty((B, E), dtype=_I32)
    tokens = logits.new_empty(B, dtype=_I32)
    mean = logits.new_empty((B, E), dtype=_F32)
    _call("ep_balance_loss", index, _balance_struct(*fields), logits.data_ptr(), topk_idx.data_ptr(),
          _ptr(seq_offsets), _ptr(token_mask), loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), mean.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return loss, counts, tokens, mean


def ep_balance_loss_backward(
    grad_loss: torch.Tensor,
    logits: torch.Tensor,
    counts: torch.Tensor,
    tokens: torch.Tensor,
    topk: int,
    score: int = _lib.EP_SCORE_SOFTMAX,
    coef: float = 1.0,
    seq_offsets: torch.Tensor | None = None,
    token_mask: torch.Tensor | None = None,
    grad_base: torch.Tensor | None = None,
    out: torch.Tensor | None = None,
) -> torch.Tensor:
    """Gradient of ``ep_balance_loss``'s loss to the logits, [T, E] in their
    type, given grad_loss (fp32 [1]), the counts and tokens that call returned
    and its other arguments; the counts are constants.  ``grad_base`` (the
    logits' type, for example ``ep_route_backward``'s) is added; ``out`` may be
    grad_base itself."""
    K = int(topk)
    T, E, B, index, fields = _balance_args(logits, K, score, coef, seq_offsets, token_mask)
    _check(counts, "counts", _I32, (B, E), index)
    _check(tokens, "tokens", _I32, (B,), index)
    _check(grad_loss, "grad_loss", _F32, None, index)
    if grad_loss.numel() != 1:
        raise ValueError("grad_loss must hold one value")
    if grad_base is not None:
        _check(grad_base, "grad_base", logits.dtype, (T, E), index)
    if out is None:
        out = torch.empty_like(logits)
    else:
        _check(out, "out", logits.dtype, (T, E), index)
    _call("ep_balance_loss_backward", index, _balance_struct(*fields), grad_loss.data_ptr(), logits.data_ptr(),
          _ptr(seq_offsets), _ptr(token_mask), counts.data_ptr(), tokens.data_ptr(), _ptr(grad_base), out.data_ptr())
    return out
