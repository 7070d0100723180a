"""GPU parity of the router and its gradient against the float64 oracle: the
choice equal index for index, weights and gradients within bounds derived in
oracle.layer_oracle."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as LO

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def ep():
    import combine_ep_layout_03_amd as m

    return m


def _score(name):
    return ep().EP_SCORE_SIGMOID if name == "sigmoid" else ep().EP_SCORE_SOFTMAX


def _logits(T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g)).to(dtype)


def _bias(E, seed, steps=True):
    g = torch.Generator().manual_seed(seed + 77)
    b = torch.randn(E, generator=g) * 0.04
    return (b * 1000).round() / 1000 if steps else b


def _check(l, K, score="softmax", bias=None, G=0, TG=0, gtop=1, renorm=False, scale=1.0, mask=None, copies=1):
    """One call on `copies` repetitions of the tokens l against the oracle on l."""
    print(f"route {copies} x {tuple(l.shape)} {l.dtype} K={K} {score} bias={bias is not None} G={G}/{TG} top{gtop} "
          f"renorm={renorm}", flush=True)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    if copies > 1:
        big = [None if t is None else t.to(DEV).repeat(copies, *[1] * (t.dim() - 1)) for t in (l, mask)]
        idx, w = ep().ep_route(big[0], K, score=_score(score), bias=dev(bias), num_groups=G, topk_groups=TG,
                               group_top=gtop, renormalize=renorm, scale=scale, token_mask=big[1])
        one = idx[: len(l)].repeat(copies, 1), w[: len(l)].repeat(copies, 1)
        assert torch.equal(idx, one[0]) and torch.equal(w, one[1])
        idx, w = idx[: len(l)], w[: len(l)]
        return _compare(l, K, score, bias, G, TG, gtop, renorm, scale, mask, idx, w)
    idx, w = ep().ep_route(dev(l), K, score=_score(score), bias=dev(bias), num_groups=G, topk_groups=TG,
                           group_top=gtop, renormalize=renorm, scale=scale, token_mask=dev(mask))
    torch.cuda.synchronize()
    return _compare(l, K, score, bias, G, TG, gtop, renorm, scale, mask, idx, w)


def _compare(l, K, score, bias, G, TG, gtop, renorm, scale, mask, idx, w):
    l64 = l.double().numpy()
    want_i, want_w = LO.route(l64, K, score, None if bias is None else bias.double().numpy(), G, TG, gtop, renorm, scale,
                              None if mask is None else mask.numpy())
    got_i, got_w = idx.cpu().numpy(), w.cpu().double().numpy()
    assert np.array_equal(got_i, want_i), np.argwhere(got_i != want_i)[:4]
    sel = want_i >= 0
    assert (got_w[~sel] == 0).all()
    # among fp32's denormals steps are absolute: the exponential is off by up to
    # 2^-149, the quotient by 2^-150, both times scale, and the product by 2^-150
    tiny = 2.0**-148 * max(1.0, scale)
    assert (np.abs(got_w - want_w) <= LO.weights_rtol(l64, want_i) * np.abs(want_w) + tiny).all()
    return idx, w


# (T, E, K): one token, odd sizes, every kernel variant (up to 64, 128, 256, 512, 1024 experts), K to 32
SHAPES = [(1, 1, 1), (1, 256, 8), (3, 7, 3), (5, 64, 4), (4, 65, 6), (33, 128, 8), (17, 129, 2), (64, 256, 8),
          (7, 257, 9), (6, 512, 17), (5, 513, 32), (9, 1024, 32), (2, 60, 32)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_shapes(T, E, K, dtype):
    l = _logits(T, E, dtype, T * 31 + E)
    _check(l, K)
    _check(l, K, "softmax", renorm=True, scale=2.5)
    _check(l, K, "sigmoid", bias=_bias(E, T), renorm=True)
    _check(l, K, "softmax", bias=_bias(E, T, steps=False) * 0.1)
    _check(l, K, "sigmoid")


# more than 2048 tokens: 16, 32 or 64 lanes a token, 4 to 16 values a lane, all or half of them kept
BIG = [(3, 1, 1), (37, 7, 3), (33, 64, 32), (21, 100, 9), (41, 128, 8), (35, 129, 8), (29, 256, 8), (13, 256, 17),
       (27, 255, 8), (19, 300, 8), (11, 512, 32), (17, 512, 5), (9, 1024, 8), (7, 1000, 32)]


@pytest.mark.parametrize("T,E,K", BIG)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_large_batches(T, E, K, dtype):
    l = _logits(T, E, dtype, T * 7 + E)
    copies = 2100 // T + 1
    _check(l, K, renorm=True, scale=2.5, copies=copies)
    _check(l, K, "softmax", copies=copies)
    _check(l, K, "sigmoid", bias=_bias(E, T), copies=copies)
    _check(l, K, "softmax", bias=_bias(E, T, steps=False) * 0.1, renorm=True, copies=copies)
    if E % 4 == 0:
        G = 4 if E <= 512 else 8
        TG = next(n for n in range(1, G + 1) if n * E // G >= K)
        mask = torch.ones(T, dtype=torch.bool)
        mask[::3] = False
        _check(l, K, "sigmoid", _bias(E, G), G, TG, 2, True, 2.5, mask, copies=copies)
        _check(l, K, "softmax", None, G, TG, 2, copies=copies)
        _check(l, K, "softmax", None, G, TG, 1, mask=mask, copies=copies)


@pytest.mark.parametrize("E,G,TG,gtop,K", [(256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (160, 8, 3, 2, 6), (96, 32, 5, 2, 7),
                                           (64, 64, 9, 2, 9), (12, 1, 1, 2, 12), (1024, 64, 2, 2, 32), (70, 7, 7, 1, 5),
                                           (768, 3, 2, 2, 10)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_groups(E, G, TG, gtop, K, dtype):
    l = _logits(37, E, dtype, E + G)
    _check(l, K, "sigmoid", _bias(E, G), G, TG, gtop, True, 2.5)
    _check(l, K, "softmax", None, G, TG, gtop)
    _check(l, K, "softmax", _bias(E, G) * 0.05, G, TG, gtop, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_masks_and_special_values(dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    T, E = 24, 40
    l = _logits(T, E, dtype, 9)
    l[0] = -inf  # nothing left
    l[1] = nan
    l[2, 3:] = -inf  # fewer than K
    l[3] = low  # the type's lowest value everywhere: equal finite logits
    l[4, :30] = low
    l[5, 7] = inf
    l[6, 7] = l[6, 3] = inf
    l[7, ::2] = nan
    l[8] = 0.0
    l[8, 5] = -0.0  # equals +0: the lowest index goes first
    l[9, :] = 100.0
    l[10, :] = -100.0
    l[11] *= 30
    l[12, 0] = torch.finfo(dtype).max
    l[12, 1] = inf
    mask = torch.ones(T, dtype=torch.bool)
    mask[[13, 20, 23]] = False
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            for n in (1, 90):
                _check(l, 6, score, renorm=renorm, mask=mask, copies=n)
                _check(l, 6, score, bias=_bias(E, 3), renorm=renorm, mask=mask, copies=n)
                _check(l, 6, score, bias=torch.zeros(E), G=8, TG=3, gtop=2, renorm=renorm, mask=mask, copies=n)
    b = _bias(E, 4)
    b[0], b[1], b[2] = nan, -inf, inf
    _check(l[13:], 6, "sigmoid", bias=b)
    u8 = mask.to(torch.uint8)
    a = ep().ep_route(l.to(DEV), 4, token_mask=u8.to(DEV))
    c = ep().ep_route(l.to(DEV), 4, token_mask=mask.to(DEV))
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_route_neighbouring_scores_are_ordered_in_binary64():
    """Logits and biases whose fp32 scores tie or cross although their binary64
    values do not: a permutation of experts whose score + bias differ by less
    than an fp32 step of the score."""
    T, E = 32, 64
    rng = np.random.default_rng(2)
    l = torch.from_numpy(rng.uniform(-1, 1, (T, E)).astype(np.float32))
    s = 1 / (1 + np.exp(-l.double().numpy()))
    # biases that bring every score of token 0 to nearly the same sum
    b = torch.from_numpy((0.9 - s[0]).astype(np.float32))
    l = l[:1].repeat(T, 1) + torch.from_numpy(rng.integers(-3, 4, (T, E)).astype(np.float32)) * 2.0**-24
    _check(l, 8, "sigmoid", bias=b)
    _check(l, 32, "sigmoid", bias=b, renorm=True)
    _check(l, 8, "sigmoid", bias=b, G=8, TG=3, gtop=2)
    _check(l, 8, "sigmoid", bias=torch.zeros(E), G=8, TG=3, gtop=2)
    p = torch.softmax(l[0].double(), 0)
    _check(l, 8, "softmax", bias=(0.5 - p).float())
    for n in (8, 32):
        _check(l, n, "sigmoid", bias=b, renorm=True, copies=70)
        _check(l, n, "softmax", bias=(0.5 - p).float(), copies=70)
        _check(l, n, copies=70)  # fp32 logits a step apart
    _check(l, 8, "sigmoid", bias=b, G=8, TG=3, gtop=2, copies=70)
    _check(l, 8, "softmax", G=8, TG=3, gtop=2, copies=70)


def test_route_all_experts_equal():
    """Every value equal (a router that starts at zero): more candidates than
    are kept, ties to the lowest index."""
    for E in (64, 256, 1024):
        for copies in (1, 1100):
            l = torch.zeros(2, E)
            _check(l, 8, copies=copies)
            _check(l, 8, "sigmoid", bias=torch.zeros(E), G=4, TG=2, gtop=2, renorm=True, copies=copies)


@pytest.mark.parametrize("E", [64, 256, 512, 1000])
@pytest.mark.parametrize("K", [1, 8, 17, 32])
def test_route_ties_and_experts_of_one_lane(E, K):
    """fp32 logits with more equal ones than are kept as candidates, across the
    Kth place and above it, with NaN and -inf between them, and with the
    largest ones all held by one lane."""
    g = torch.Generator().manual_seed(E + K)
    l = torch.randn(10, E, generator=g)
    l[0] = 0.25
    l[1, ::3], l[1, 1::3] = float("nan"), 1.0
    l[2, : E // 2] = float("-inf")
    l[2, E // 2:] = -2.5
    l[3] = torch.where(torch.rand(E, generator=g) < 0.5, 3.0, l[3])
    l[4, torch.randperm(E, generator=g)[: K - 1]] = 9.0
    l[4, torch.randperm(E, generator=g)[: E // 2]] = 4.0
    for i, lanes in enumerate((16, 32, 64)):  # lane 3's experts of 16, 32 or 64 lanes a token
        held = [e for e in range(E) if e // 4 % lanes == 3]
        l[5 + i, held] += 10.0
    l[8] = l[8].to(torch.bfloat16).float()
    l[9, 1:] = float("nan")
    for copies in (1, 230):
        _check(l, K, copies=copies)
        _check(l, K, "sigmoid", renorm=True, copies=copies)
        if E % 8 == 0 and K <= E // 4:
            _check(l, K, G=8, TG=3, copies=copies)
            _check(l, K, G=8, TG=3, gtop=2, copies=copies)


def test_route_offsets_past_32_bits():
    """9 million tokens x 256 bf16 logits, 4.6 GB: the last tokens as in a call
    of their own, and the gradient likewise."""
    m = ep()
    T, E, K = 9_000_000, 256, 8
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    l[-300:] = _logits(300, E, torch.bfloat16, 3).to(DEV)
    idx, w = m.ep_route(l, K, renormalize=True)
    one = l[-300:].clone()
    want = m.ep_route(one, K, renormalize=True)
    assert torch.equal(idx[-300:], want[0]) and torch.equal(w[-300:], want[1])
    assert torch.equal(idx[0], torch.arange(K, device=DEV))
    g = m.ep_route_backward(w, l, idx)
    assert torch.equal(g[-300:], m.ep_route_backward(want[1], one, want[0]))


def test_route_noncontiguous_alignment_and_out():
    """Logits at an address of element alignment only, rows of a length that
    is no multiple of a vector; outputs written in place."""
    m = ep()
    flat = _logits(1, 33 * 64 + 1, torch.float32, 5).to(DEV).reshape(-1)
    l = flat[1:].reshape(33, 64)
    idx, w = m.ep_route(l, 8)
    out = (torch.full((33, 8), 99, dtype=torch.int64, device=DEV), torch.full((33, 8), 9.0, device=DEV))
    got = m.ep_route(l.clone(), 8, out=out)
    assert got[0] is out[0] and torch.equal(idx, out[0]) and torch.equal(w, out[1])
    with pytest.raises(ValueError, match="contiguous"):
        m.ep_route(l.t(), 8)
    with pytest.raises(m.EPError):
        m.ep_route(l, 65)
    i0, w0 = m.ep_route(l[:0], 8)
    assert i0.shape == (0, 8) and w0.shape == (0, 8)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 7, 3), (65, 64, 4), (9, 130, 8), (20, 256, 8), (5, 300, 20),
                                   (4, 1024, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, K, dtype, score, renorm):
    l = _logits(T, E, dtype, T + E)
    l[0, 0] = -float("inf")
    l[-1, E // 2] = 30.0
    idx, _ = LO.route(l.double().numpy(), K, score, renorm=renorm)
    if T > 3:
        idx[1] = -1  # a token without a selection
        idx[2, 0] = E + 5  # out of range: no part
        idx[3, K - 1] = idx[3, 0]  # named twice
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(K))
    got = ep().ep_route_backward(g.to(DEV), l.to(DEV), torch.from_numpy(idx).to(DEV), score=_score(score),
                                 renormalize=renorm, scale=1.5)
    assert got.dtype == dtype and got.shape == l.shape
    want, bound = LO.route_backward(g.double().numpy(), l.double().numpy(), idx, score, renorm, 1.5)
    if dtype == torch.bfloat16:
        bound = bound + LO.UBF * np.abs(want)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= bound + 2.0**-133).all(), (err - bound).max()


def test_route_backward_masked_rows_are_zero():
    m = ep()
    l = torch.full((4, 10), -float("inf"), device=DEV)
    l[1] = float("nan")
    l[2, 4] = 1.0
    idx = torch.tensor([[-1, -1], [3, 2], [4, -1], [0, 4]], device=DEV)
    g = torch.ones(4, 2, device=DEV)
    for score in (m.EP_SCORE_SOFTMAX, m.EP_SCORE_SIGMOID):
        for renorm in (False, True):
            got = m.ep_route_backward(g, l, idx, score=score, renormalize=renorm)
            got[2, 4] = 0.0  # the only selection that can have a gradient
            assert (got == 0).all()


def test_route_graph_and_streams():
    """Captured and replayed on new logits, against eager calls in between;
    two calls at once on two streams."""
    m = ep()
    l, b, g = _logits(200, 256, torch.float32, 1).to(DEV), _bias(256, 1).to(DEV), torch.randn(3000, 8, device=DEV)
    kw = dict(score=m.EP_SCORE_SIGMOID, renormalize=True, scale=2.0)

    def step(x):
        idx, w = m.ep_route(x, 8, bias=b, num_groups=8, topk_groups=4, group_top=2, **kw)
        return idx, w, m.ep_route_backward(g[: len(x)], x, idx, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(l)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(l)
    for rep in range(4):
        l.copy_(_logits(200, 256, torch.float32, 50 + rep))
        want = step(l.clone())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(res, want))
    other = _logits(3000, 256, torch.float32, 7).to(DEV)
    want_l, want_o = step(l), step(other)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got_o = step(other)
    got_l = step(l)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got_l + got_o, want_l + want_o))


@pytest.mark.parametrize("E", [64, 100, 256, 300, 1000])
@pytest.mark.parametrize("copies", [1, 160])
def test_route_infinite_biases(E, copies):
    """Several experts with a bias of +inf have equal selection values: the
    lowest indices go first, whichever lanes hold them, alone, beside finite
    ones, and in groups."""
    l = _logits(14, E, torch.float32, E)
    rng = np.random.default_rng(E)
    for some in ([1, 4], [E - 1, E - 2, 5, 8, 3], sorted(rng.choice(E, 24, replace=False)), range(E)):
        b = _bias(E, 5)
        b[torch.tensor(list(some))] = float("inf")
        b[0] = float("nan")
        b[2] = float("-inf")
        for K in (1, 4, 8, 32):
            _check(l, K, "sigmoid", bias=b, copies=copies)
            _check(l.to(torch.bfloat16), K, "softmax", bias=b, renorm=True, copies=copies)
        if E % 4 == 0:
            for gtop in (1, 2):
                _check(l, 3, "sigmoid", b, 4, 2, gtop, copies=copies)
                _check(l, 8, "softmax", b, E // (4 if E <= 256 else 20), 3, gtop, copies=copies)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("copies", [1, 160])
def test_route_group_values_past_fp32(sign, copies):
    """Group values that are sums of two finite biases and overflow fp32: the
    groups are still told apart, and differ from one without experts."""
    E, G = 64, 8
    l = _logits(15, E, torch.float32, 8)
    base = sign * torch.tensor([2.0e38, 2.2e38, 3.0e38, 2.9e38, 1.8e38, 3.3e38, 2.5e38, 3.4e38])
    b = base.repeat_interleave(E // G)
    for TG in (1, 3, 7):
        _check(l, 6, "sigmoid", b, G, TG, 2, copies=copies)
        _check(l, 6, "softmax", b, G, TG, 2, copies=copies)
    b[8:16] = float("-inf")  # a group without an expert to choose
    b[16:24] = float("nan")
    for TG in (2, 6, 8):
        _check(l, 6, "sigmoid", b, G, TG, 2, copies=copies)
    b[24] = float("inf")
    _check(l, 6, "sigmoid", b, G, 2, 2, copies=copies)
    b = torch.full((E,), sign * 3.0e38)  # all equal, all past fp32
    _check(l, 6, "sigmoid", b, G, 3, 2, copies=copies)
