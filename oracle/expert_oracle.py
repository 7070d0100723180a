"""CPU oracle of the experts' layers and the balance loss.

Plain numpy in float64, one expert or one token at a time, written from the
formulas and sharing nothing with the HIP kernels.  bf16 inputs arrive as
float64 values.  The bounds are absolute errors per element for a kernel that
accumulates in fp32 and rounds once to its output type.
"""
from __future__ import annotations

import math

import numpy as np

from .layer_oracle import U32, UBF, _clean

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
TINY = 2.0**-120  # what fp32 may lose to denormals on the way
_K = math.sqrt(2 / math.pi)
_C = 0.044715
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sig(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def act(z, kind):
    """(value, derivative, error of the value, of the derivative) in fp32.

    An exponential's argument x is off by a step or two relative, so exp(x) by
    2 |x| half steps, and what is formed from it by at most 40 more; 1 - p is
    off by half a step of 1."""
    if kind == "none":
        return z, np.ones_like(z), np.zeros_like(z), np.zeros_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(float), np.zeros_like(z), np.zeros_like(z)
    if kind == "silu":
        p, q = _sig(z), _sig(-z)
        size = p + np.abs(z) * p * q
        v, d, x = z * p, p + z * p * q, np.abs(z)
        lost = 2 * np.abs(z) * p
    elif kind == "gelu":
        p = 0.5 * _erfc(-z / math.sqrt(2))
        phi = np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        size = p + np.abs(z) * phi
        v, d, x = z * p, p + z * phi, z * z
        lost = 0.0
    else:
        u = _K * (z + _C * z**3)
        p, q = _sig(2 * u), _sig(-2 * u)
        grow = 2 * np.abs(z) * _K * (1 + 3 * _C * z * z)
        size = p + grow * p * q
        v, d, x = z * p, p + np.sign(z) * grow * p * q, 4 * np.abs(u)
        lost = 2 * grow * p
    ev = (4 * x + 40) * U32 * np.abs(v) + TINY
    ed = U32 * ((4 * x + 60) * size + lost) + TINY
    return v, d, ev, ed


def linear(x, w, bias, kind, gated, residual, rows_of):
    """rows_of: per expert (rows of x, receive rows).  Returns (out, its bound,
    pre, its bound), NaN where no selection is."""
    E, W, H = w.shape
    N = W // 2 if gated else W
    R = max((int(o.max()) + 1 for _, o in rows_of if len(o)), default=0) if residual is None else residual.shape[0]
    out, pre = np.full((R, N), np.nan), np.full((R, W), np.nan)
    bout, bpre = out.copy(), pre.copy()
    for e, (xi, oi) in enumerate(rows_of):
        if len(xi) == 0:
            continue
        z = x[xi] @ w[e].T
        dz = H * U32 * (np.abs(x[xi]) @ np.abs(w[e]).T)
        if bias is not None:
            z = z + bias[e]
            dz = dz + 2 * U32 * (np.abs(z) + np.abs(bias[e]))
        pre[oi], bpre[oi] = z, UBF * np.abs(z) + 2 * dz
        v, _, ev, _ = act(z[:, :N], kind)
        ev = ev + 1.2 * dz[:, :N]  # no activation is steeper
        if gated:
            u, du = z[:, N:], dz[:, N:]
            ev = np.abs(u) * ev + np.abs(v) * du + ev * du + U32 * np.abs(u * v)
            v = u * v
        if residual is not None:
            v = v + residual[oi]
            ev = ev + 2 * U32 * (np.abs(v) + np.abs(residual[oi]))
        out[oi], bout[oi] = v, UBF * np.abs(v) + 2 * ev
    return out, bout, pre, bpre


def grad_pre(go, pre, kind, gated):
    """(grad_pre, its bound) for the rows given."""
    N = go.shape[1]
    v, d, ev, ed = act(pre[:, :N], kind)
    if gated:
        u = pre[:, N:]
        g = np.concatenate([go * u * d, go * v], 1)
        b = np.concatenate([np.abs(go * u) * (ed + 2 * U32 * np.abs(d)), np.abs(go) * (ev + U32 * np.abs(v))], 1)
    else:
        g, b = go * d, np.abs(go) * (ed + U32 * np.abs(d))
    return g, UBF * np.abs(g) + 2 * b + TINY


def linear_backward(g, x, w, rows_of):
    """From g = grad_pre as it was rounded: ((grad_x, bound), (grad_w, bound),
    (grad_bias, bound)); grad_x is NaN where no selection is."""
    E, W, H = w.shape
    gx, bx = np.full((g.shape[0], H), np.nan), np.full((g.shape[0], H), np.nan)
    gw, bw = np.zeros(w.shape), np.zeros(w.shape)
    gb, bb = np.zeros((E, W)), np.zeros((E, W))
    for e, (xi, oi) in enumerate(rows_of):
        n = len(xi)
        if n == 0:
            continue
        gx[oi] = g[oi] @ w[e]
        bx[oi] = UBF * np.abs(gx[oi]) + 2 * W * U32 * (np.abs(g[oi]) @ np.abs(w[e]))
        gw[e] = g[oi].T @ x[xi]
        bw[e] = UBF * np.abs(gw[e]) + 2 * n * U32 * (np.abs(g[oi]).T @ np.abs(x[xi]))
        gb[e] = g[oi].sum(0)
        bb[e] = UBF * np.abs(gb[e]) + 2 * n * U32 * np.abs(g[oi]).sum(0)
    return (gx, bx), (gw, bw), (gb, bb)


def share(l, score):
    """(scores over their sum, 1 - score) of one token's cleaned logits."""
    if not np.isfinite(l).any():
        return np.zeros_like(l), np.ones_like(l)
    if score == "softmax":
        e = np.exp(l - l.max())
        return e / e.sum(), np.ones_like(l)
    top = min(float(l.max()), 0.0)
    with np.errstate(over="ignore"):
        s = np.where(l >= 0, _sig(l), np.exp(np.minimum(l, 0) - top) * _sig(-np.minimum(l, 0)))
        return s / s.sum(), _sig(-l)


def _tokens(T, seq, mask):
    seq = [0, T] if seq is None else list(seq)
    for b in range(len(seq) - 1):
        yield b, [t for t in range(seq[b], seq[b + 1]) if mask is None or mask[t]]


def balance(logits, idx, score, coef, seq=None, mask=None):
    """loss, counts, tokens, mean."""
    T, E = logits.shape
    K, B = idx.shape[1], 1 if seq is None else len(seq) - 1
    loss, counts = 0.0, np.zeros((B, E), np.int64)
    tokens, mean = np.zeros(B, np.int64), np.zeros((B, E))
    for b, at in _tokens(T, seq, mask):
        tokens[b] = len(at)
        for t in at:
            mean[b] += share(_clean(np.asarray(logits[t], np.float64)), score)[0]
            for e in idx[t]:
                if 0 <= e < E:
                    counts[b, e] += 1
        if at:
            mean[b] /= len(at)
            loss += coef / B * E / (K * len(at)) * (counts[b] * mean[b]).sum()
    return loss, counts, tokens, mean


def share_rtol(logits):
    """Relative error of a share: exponentials of arguments off by half a step
    of the largest logit or difference (twice, for the two of a sigmoid), and
    sums of up to 16 values a lane and 6 levels."""
    big = np.where(np.isfinite(logits), np.abs(logits), 0.0).max(initial=0.0)
    return (8 * big + 64) * U32


def balance_backward(g, logits, counts, tokens, K, score, coef, seq=None, mask=None, base=None):
    """(grad_logits, bound without the output's rounding)."""
    T, E = logits.shape
    out = np.zeros((T, E)) if base is None else base.astype(np.float64).copy()
    bound = 2 * U32 * np.abs(out)
    for b, at in _tokens(T, seq, mask):
        for t in at:
            p, rest = share(_clean(np.asarray(logits[t], np.float64)), score)
            f = g * coef * E / (K * counts.shape[0] * float(tokens[b]) ** 2) * counts[b]
            out[t] += p * rest * (f - (f * p).sum())
            bound[t] += 4 * share_rtol(logits[t]) * p * rest * (np.abs(f) + (np.abs(f) * p).sum())
    return out, bound + 2 * U32 * np.abs(out) + TINY
