"""Pins of the expert oracle: its gradients against central differences of its
forward formulas in float64, activations against closed values (CPU only)."""
import math

import numpy as np
import pytest

from oracle import expert_oracle as XO


def _diff(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += eps
        lo[i] -= eps
        g[i] = (f(hi) - f(lo)) / (2 * eps)
    return g


@pytest.mark.parametrize("kind", XO.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_linear_backward_matches_differences(kind, gated):
    rng = np.random.default_rng(7)
    H, N, E = 5, 4, 3
    W = 2 * N if gated else N
    x, go = rng.standard_normal((6, H)), rng.standard_normal((7, N))
    w, b = rng.standard_normal((E, W, H)), rng.standard_normal((E, W))
    res = rng.standard_normal((7, N))
    # expert 1 has no row; x rows are gathered, one of them twice
    rows = [(np.array([0, 3]), np.array([0, 1])), (np.array([], int), np.array([], int)),
            (np.array([5, 1, 3]), np.array([2, 3, 5]))]
    _, _, pre, _ = XO.linear(x, w, b, kind, gated, res, rows)
    at = np.concatenate([o for _, o in rows])
    g = np.zeros((7, W))
    g[at] = XO.grad_pre(go[at], pre[at], kind, gated)[0]
    (gx, _), (gw, _), (gb, _) = XO.linear_backward(g, x, w, rows)
    # a token's gradient is the sum of its rows'
    total = np.zeros_like(x)
    for xi, oi in rows:
        for i, o in zip(xi, oi):
            total[i] += gx[o]

    def loss(x_, w_, b_):
        return (go[at] * XO.linear(x_, w_, b_, kind, gated, res, rows)[0][at]).sum()

    assert np.abs(total - _diff(lambda v: loss(v, w, b), x)).max() < 1e-7
    assert np.abs(gw - _diff(lambda v: loss(x, v, b), w)).max() < 1e-7
    assert np.abs(gb - _diff(lambda v: loss(x, w, v), b)).max() < 1e-7
    assert np.isnan(gx[[4, 6]]).all() and (gw[1] == 0).all() and (gb[1] == 0).all()


def test_activations_by_hand():
    z = np.array([-2.0, 0.0, 1.0])
    assert XO.act(z, "relu")[0].tolist() == [0, 0, 1] and XO.act(z, "relu")[1].tolist() == [0, 0, 1]
    assert XO.act(z, "silu")[0] == pytest.approx([-2 / (1 + math.e**2), 0, 1 / (1 + math.exp(-1))], abs=1e-15)
    assert XO.act(z, "gelu")[0] == pytest.approx([-2 * 0.022750131948179, 0, 0.841344746068543], abs=1e-13)
    t = math.tanh(math.sqrt(2 / math.pi) * 1.044715)
    assert XO.act(z, "gelu_tanh")[0][2] == pytest.approx(0.5 * (1 + t), abs=1e-15)
    assert XO.act(z, "gelu")[1][1] == 0.5 and XO.act(z, "gelu_tanh")[1][1] == 0.5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_backward_matches_differences(score):
    rng = np.random.default_rng(8)
    T, E, K = 9, 5, 2
    l = rng.standard_normal((T, E)) * 2
    idx = np.argsort(-l, axis=1)[:, :K].copy()
    idx[4, 1] = -1
    seq, mask = [1, 4, 4, 8], np.array([1, 1, 0, 1, 1, 1, 1, 1, 1], bool)
    loss, counts, tokens, mean = XO.balance(l, idx, score, 0.5, seq, mask)
    assert tokens.tolist() == [2, 0, 4] and counts.sum() == 2 * 6 - 1 and (mean[1] == 0).all()
    assert mean[0].sum() == pytest.approx(1, abs=1e-14)
    base = rng.standard_normal((T, E))
    got, _ = XO.balance_backward(1.5, l, counts, tokens, K, score, 0.5, seq, mask, base)
    want = _diff(lambda v: 1.5 * XO.balance(v, idx, score, 0.5, seq, mask)[0], l)
    assert np.abs(got - base - want).max() < 1e-8
    assert (got[[0, 2, 8]] == base[[0, 2, 8]]).all()


def test_balance_of_a_balanced_router_is_coef():
    l = np.zeros((8, 4))
    idx = np.array([[0], [1], [2], [3]] * 2)
    for score in ("softmax", "sigmoid"):
        assert XO.balance(l, idx, score, 0.25)[0] == pytest.approx(0.25, abs=1e-15)
    # scores that underflow fp32, and ones that are out, still have shares
    p, rest = XO.share(np.array([-300.0, -300.0, -np.inf]), "sigmoid")
    assert p == pytest.approx([0.5, 0.5, 0], abs=1e-12) and rest.tolist() == [1, 1, 1]
    assert XO.share(np.full(3, -np.inf), "softmax")[0].tolist() == [0, 0, 0]
