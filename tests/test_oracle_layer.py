"""Pins of the layer oracle (router, gradients, adapters): the gradients
against central differences of the forward formulas in float64, and the
router's ties and masks by hand (CPU only)."""
import numpy as np
import pytest

from oracle import layer_oracle as LO


def _diff(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += eps
        lo[i] -= eps
        g[i] = (f(hi) - f(lo)) / (2 * eps)
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_matches_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, E, K = 4, 7, 3
    l, g = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    idx, _ = LO.route(l, K, score, renorm=renorm, scale=1.7)
    idx[1, 2] = -1
    idx[2] = -1

    def loss(x):
        total = 0.0
        for t in range(T):
            ks = [k for k in range(K) if idx[t, k] >= 0]
            if ks:
                w = LO.chosen_weights(x[t], idx[t, ks], score, renorm)
                total += (g[t, ks] * w * 1.7).sum()
        return total

    got, _ = LO.route_backward(g, l, idx, score, renorm, 1.7)
    # second-order differences: error of order eps^2 plus rounding 1e-16 / eps
    assert np.abs(got - _diff(loss, l)).max() < 1e-8


def test_lora_backward_matches_differences():
    rng = np.random.default_rng(4)
    H, N, R, E = 6, 5, 3, 3
    x, go = rng.standard_normal((7, H)), rng.standard_normal((7, N))
    a, b, s = rng.standard_normal((E, R, H)), rng.standard_normal((E, N, R)), rng.standard_normal(E)
    rows = [(np.array([0, 3]), np.array([0, 3])), (np.array([], int), np.array([], int)),
            (np.array([5, 1, 6]), np.array([5, 1, 6]))]
    base = np.zeros((7, N))
    (gx, _), (ga, _), (gb, _) = LO.lora_backward(go, x, a, b, s, np.zeros((7, H)), rows)

    def loss(x_, a_, b_):
        return (go * LO.lora(x_, a_, b_, s, base, rows)[0]).sum()

    assert np.abs(gx - _diff(lambda v: loss(v, a, b), x)).max() < 1e-7
    assert np.abs(ga - _diff(lambda v: loss(x, v, b), a)).max() < 1e-7
    assert np.abs(gb - _diff(lambda v: loss(x, a, v), b)).max() < 1e-7
    assert (gx[2] == 0).all() and (ga[1] == 0).all()


def test_combine_backward_matches_differences():
    rng = np.random.default_rng(5)
    slot = np.array([[0, 2], [-1, 1], [3, 9]])
    w = rng.standard_normal((3, 2)).astype(np.float32)
    y, go = rng.standard_normal((4, 5)), rng.standard_normal((3, 5))

    def loss(y_, w_):
        return sum(w_[t, k] * (go[t] * y_[slot[t, k]]).sum() for t in range(3) for k in range(2)
                   if 0 <= slot[t, k] < 4)

    gy, gw, _ = LO.combine_backward(go, y, slot, w)
    assert np.abs(np.nan_to_num(gy) - _diff(lambda v: loss(v, w.astype(float)), y)).max() < 1e-6
    assert np.abs(gw - _diff(lambda v: loss(y, v), w.astype(float))).max() < 1e-8


def test_route_ties_masks_and_groups_by_hand():
    inf, nan = np.inf, np.nan
    l = np.array([[1, 2, 2, 0.0], [nan, -inf, 3, -inf], [-inf] * 4, [inf, 5, inf, 0]])
    idx, w = LO.route(l, 2)
    assert idx.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert w[1].tolist() == [1, 0] and w[2].tolist() == [0, 0] and w[3].tolist() == [0.5, 0.5]
    # a bias takes part in the choice, not in the weight
    idx, w = LO.route(l[:1], 1, "sigmoid", bias=np.array([0, 0, 0, 5.0]))
    assert idx.tolist() == [[3]] and w.tolist() == [[0.5]]
    # groups {0,1} and {2,3}: best of each 2 and 2: the first stays open; sums 3 > 2
    idx, _ = LO.route(l[:1], 2, G=2, TG=1)
    assert idx.tolist() == [[1, 0]]
    idx, _ = LO.route(np.array([[1, 2, 3.5, -9]]), 2, "sigmoid", bias=np.zeros(4), G=2, TG=1, gtop=2)
    assert idx.tolist() == [[1, 0]]
    idx, w = LO.route(l[:1], 2, mask=[0])
    assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]]
