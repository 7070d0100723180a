"""CPU oracle of the layer operators (router, gradients, low-rank adapters).

Plain numpy in float64, one token or one expert at a time, written from the
formulas and sharing nothing with the HIP kernels.  bf16 inputs arrive as
float64 values.  The ``*_bound`` results are absolute error bounds per
element for a kernel that accumulates in fp32, holds the adapters' inner
products in fp32 and rounds once to its output type.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0**-24  # half a step of fp32, relative
UBF = 2.0**-8  # half a step of bf16, relative


def _clean(l):
    """NaN -> -inf; +inf -> the largest finite fp32."""
    l = np.where(np.isnan(l), -np.inf, l)
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(l, score):
    """Scores of one token's cleaned logits; 0 where a logit is -inf."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        if not np.isfinite(l).any():
            return np.zeros_like(l)
        e = np.exp(l - l.max())
        return e / e.sum()


def _order(values):
    """Indices by descending value, equal values by ascending index, without
    the -inf ones."""
    return [int(i) for i in sorted(range(len(values)), key=lambda i: (-values[i], i)) if values[i] > -np.inf]


def chosen_weights(l, idx, score, renorm):
    """Scores of the chosen logits (idx without -1), optionally over their sum."""
    s = scores(l, score)[idx]
    if not renorm:
        return s
    if score == "softmax":
        e = np.exp(l[idx] - l[idx].max())
    else:
        logs = np.minimum(l[idx], 0) - np.log1p(np.exp(-np.abs(l[idx])))
        e = np.exp(logs - logs.max())
    return e / e.sum()


def route(logits, K, score="softmax", bias=None, G=0, TG=0, gtop=1, renorm=False, scale=1.0, mask=None):
    T, E = logits.shape
    idx = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        l = _clean(np.asarray(logits[t], np.float64))
        out = np.isneginf(l)
        s = scores(l, score)
        value = l.copy() if bias is None else s + bias
        value[np.isnan(value)] = -np.inf
        value[out] = -np.inf
        if G:
            gv = value if bias is not None or gtop == 1 else np.where(out, -np.inf, s)
            n = E // G
            total = []
            for g in range(G):
                best = sorted((v for v in gv[g * n:(g + 1) * n] if v > -np.inf), reverse=True)[:gtop]
                total.append(sum(best) if best else -np.inf)
            opened = sorted(range(G), key=lambda g: (-total[g], g))[:TG]
            for g in range(G):
                if g not in opened:
                    value[g * n:(g + 1) * n] = -np.inf
        pick = _order(value)[:K]
        if pick:
            idx[t, : len(pick)] = pick
            w[t, : len(pick)] = scale * chosen_weights(l, np.array(pick), score, renorm)
    return idx, w


def weights_rtol(logits, idx):
    """Relative error of a weight: an exponential's argument is off by half a
    step of each logit or difference that forms it (at most four of the
    largest), everything after (exponentials, a sum of up to 1024 terms over
    16 values a lane and 6 levels, quotient, scale) by at most 64 half steps."""
    big = np.where(np.isfinite(logits), np.abs(logits), 0.0).max(axis=1, initial=0.0, keepdims=True)
    return (4 * big + 64) * U32  # per token


def route_backward(gw, logits, idx, score="softmax", renorm=False, scale=1.0):
    """(grad_logits, bound without the output's rounding)."""
    T, E = logits.shape
    K = idx.shape[1]
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        l = _clean(np.asarray(logits[t], np.float64))
        ks = [k for k in range(K) if 0 <= idx[t, k] < E and l[idx[t, k]] > -np.inf]
        if not ks and not (score == "softmax" and not renorm):
            continue
        at = np.array([idx[t, k] for k in ks], int)
        g = np.array([gw[t, k] * scale for k in ks])
        s = scores(l, score)
        if renorm:
            w = chosen_weights(l, at, score, True)
            d = w * (g - (w * g).sum())
            a = w * (np.abs(g) + (w * np.abs(g)).sum())
            if score == "sigmoid":
                d, a = d / (1 + np.exp(l[at])), a / (1 + np.exp(l[at]))
            for i, e in enumerate(at):
                out[t, e] += d[i]
                bound[t, e] += a[i]
        elif score == "sigmoid":
            for i, e in enumerate(at):
                v = g[i] * s[e] / (1 + np.exp(l[e]))
                out[t, e] += v
                bound[t, e] += abs(v)
        else:
            full, mag = np.zeros(E), np.zeros(E)
            for i, e in enumerate(at):
                full[e] += g[i]
                mag[e] += abs(g[i])
            out[t] = s * (full - (s * full).sum())
            bound[t] = s * (mag + (s * mag).sum())
    # a score's relative error as in weights_rtol, twice (weight and dot)
    return out, bound * 2 * weights_rtol(logits, idx)


def combine_backward(go, y, slot, w):
    """grad_y as float32 products (before their bf16 rounding; NaN where no
    selection writes), grad_weights and its bound."""
    T, K = slot.shape
    H = go.shape[1]
    gy = np.full((y.shape[0], H), np.nan, np.float32)
    gw, bound = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = slot[t, k]
            if r < 0 or r >= y.shape[0]:
                continue
            gy[r] = np.float32(w[t, k]) * go[t].astype(np.float32)
            gw[t, k] = (go[t] * y[r]).sum()
            # a lane adds at most H / 64 + 8 products in turn, then 6 + 2 levels
            bound[t, k] = (H / 64 + 16) * U32 * np.abs(go[t] * y[r]).sum()
    return gy, gw, bound


def lora(x, a, b, scales, base, rows_of):
    """rows_of: per expert (rows of x, rows of base and out).  Returns out
    (base where no row is) and the bound."""
    out = base.copy()
    bound = np.zeros_like(out)
    H, R = x.shape[1], a.shape[1]
    for e, (xi, oi) in enumerate(rows_of):
        if len(xi) == 0:
            continue
        u = x[xi] @ a[e].T
        uerr = H * U32 * (np.abs(x[xi]) @ np.abs(a[e]).T)
        d = scales[e] * (u @ b[e].T)
        mag = abs(scales[e]) * (np.abs(u) @ np.abs(b[e]).T)
        out[oi] = base[oi] + d
        bound[oi] = (UBF * np.abs(out[oi]) + abs(scales[e]) * (uerr @ np.abs(b[e]).T) +
                     2 * (R + 2) * U32 * mag + 2 * U32 * np.abs(base[oi]))
    return out, bound


def lora_backward(go, x, a, b, scales, base, rows_of):
    """((grad_x, bound), (grad_a, bound), (grad_b, bound))."""
    gx, bx = base.copy(), np.zeros_like(base)
    ga, ba = np.zeros(a.shape), np.zeros(a.shape)
    gb, bb = np.zeros(b.shape), np.zeros(b.shape)
    H, N, R = x.shape[1], go.shape[1], a.shape[1]
    for e, (xi, oi) in enumerate(rows_of):
        n = len(xi)
        if n == 0:
            continue
        s = abs(scales[e])
        u, v = x[xi] @ a[e].T, go[oi] @ b[e]
        uerr = H * U32 * (np.abs(x[xi]) @ np.abs(a[e]).T)
        verr = N * U32 * (np.abs(go[oi]) @ np.abs(b[e]))
        gx[oi] = base[oi] + scales[e] * (v @ a[e])
        bx[oi] = (UBF * np.abs(gx[oi]) + s * (verr @ np.abs(a[e])) +
                  2 * (R + 2) * U32 * s * (np.abs(v) @ np.abs(a[e])) + 2 * U32 * np.abs(base[oi]))
        ga[e] = scales[e] * (v.T @ x[xi])
        ba[e] = (UBF * np.abs(ga[e]) + s * (verr.T @ np.abs(x[xi])) +
                 2 * (n + 2) * U32 * s * (np.abs(v).T @ np.abs(x[xi])))
        gb[e] = scales[e] * (go[oi].T @ u)
        bb[e] = (UBF * np.abs(gb[e]) + s * (np.abs(go[oi]).T @ uerr) +
                 2 * (n + 2) * U32 * s * (np.abs(go[oi]).T @ np.abs(u)))
    return (gx, bx), (ga, ba), (gb, bb)
