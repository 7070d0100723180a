"""GPU parity of the experts' layers (product with bias, activation, gate and
residual, and its gradients) against the float64 oracle within derived bounds,
and bit for bit where every sum is exact."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import ep_oracle as O
from oracle import expert_oracle as XO

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


def f64(t):
    return t.detach().cpu().double().numpy()


def u16(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def act_id(kind):
    m = ep()
    return dict(none=m.EP_ACT_NONE, relu=m.EP_ACT_RELU, silu=m.EP_ACT_SILU, gelu=m.EP_ACT_GELU,
                gelu_tanh=m.EP_ACT_GELU_TANH)[kind]


def marked(rows, width):
    """bf16 rows of a bit pattern that no result has (a NaN)."""
    return torch.full((rows, width), -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)


def bf(g, scale, *shape):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def rows_of(L, gather):
    counts, offsets = L.counts.cpu().numpy(), L.offsets.cpu().numpy()
    src = L.expert_row_src.cpu().numpy() if gather else None
    out = []
    for e in range(L.num_experts):
        o = np.arange(offsets[e], offsets[e] + counts[e])
        out.append((src[o] if gather else o, o))
    return out


def within(got, want, bound, what):
    ok = ~np.isnan(want)
    err = np.abs(f64(got)[ok] - want[ok])
    bad = ~(err <= bound[ok])
    assert not bad.any(), f"{what}: {bad.sum()} of {ok.sum()} out of bound, worst {np.nanmax(err - bound[ok])}"
    assert (u16(got)[~ok] == 0xFFFF).all(), f"{what}: a row of no selection was written"


def wider(t, extra):
    """The same rows in a buffer `extra` columns wider, NaN beyond."""
    if not extra:
        return t
    out = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    out[:, : t.shape[1]] = t
    return out


def check(T, K, E, H, N, kind="none", gated=False, bias=True, residual=True, gather=False, A=0, mask_p=0.1, extra=0,
          seed=0, idx=None, backward=True):
    """Forward and gradients of one layer against the oracle."""
    print(f"linear T={T} K={K} E={E} H={H} N={N} {kind} gated={gated} bias={bias} residual={residual} "
          f"gather={gather} A={A} extra={extra}", flush=True)
    m = ep()
    if idx is None:
        idx, _ = W.make_routing(W.Workload("x", T=T, H=H, K=K, E=E, mask_p=mask_p, seed=seed + T))
    L = m.ep_layout(idx.to(DEV), E, expert_alignment=A, expert_row_src=True)
    rows, wide = L.max_expert_rows(), (2 * N if gated else N)
    g = torch.Generator().manual_seed(seed + H * 3 + N)
    x = wider(bf(g, 1.0, T if gather else rows, H).to(DEV), extra)
    w, b = bf(g, H**-0.5, E, wide, H).to(DEV), bf(g, 0.5, E, wide).to(DEV) if bias else None
    res = wider(bf(g, 1.0, rows, N).to(DEV), extra) if residual else None
    out, pre = marked(rows, N + extra), marked(rows, wide + extra)
    m.ep_expert_linear(x, L, w, bias=b, activation=act_id(kind), gated=gated, residual=res, gather=gather, out=out,
                       pre=pre)
    torch.cuda.synchronize()
    who = rows_of(L, gather)
    x64, w64 = f64(x[:, :H]), f64(w)
    r64 = np.zeros((rows, N)) if res is None else f64(res[:, :N])
    want, bound, zwant, zbound = XO.linear(x64, w64, None if b is None else f64(b), kind, gated, r64, who)
    within(out[:, :N], want, bound, "out")
    within(pre[:, :wide], zwant, zbound, "pre")
    if extra:
        assert (u16(out[:, N:]) == 0xFFFF).all() and (u16(pre[:, wide:]) == 0xFFFF).all()
    # without pre the result is the same
    again = marked(rows, N)
    m.ep_expert_linear(x, L, w, bias=b, activation=act_id(kind), gated=gated, residual=res, gather=gather, out=again)
    assert np.array_equal(u16(again), u16(out[:, :N]))
    if not backward:
        return
    go = wider(bf(g, 1.0, rows, N).to(DEV), extra)
    bare = kind == "none" and not gated
    gx, gp = marked(rows, H + extra), None if bare else marked(rows, wide + extra)
    _, gw, gb, back = m.ep_expert_linear_backward(go, x, L, w, pre=None if bare else pre, activation=act_id(kind),
                                                  gated=gated, gather=gather, bias=True, grad_x=gx, grad_pre=gp)
    torch.cuda.synchronize()
    assert back is gp
    at = np.concatenate([o for _, o in who]) if rows else np.zeros(0, int)
    g64 = np.zeros((rows, wide))
    if bare:
        g64[at] = f64(go[:, :N])[at]
    else:
        full, fb = np.full((rows, wide), np.nan), np.full((rows, wide), np.nan)
        full[at], fb[at] = XO.grad_pre(f64(go[:, :N])[at], f64(pre[:, :wide])[at], kind, gated)
        within(gp[:, :wide], full, fb, "grad_pre")
        g64[at] = f64(gp[:, :wide])[at]
    (wx, bx), (ww, bw), (wb, bb) = XO.linear_backward(g64, x64, w64, who)
    within(gx[:, :H], wx, bx, "grad_x")
    within(gw, ww, bw, "grad_w")
    within(gb, wb, bb, "grad_bias")


# one token, odd sizes, every height of a tile, several tiles an expert,
# padding rows, experts without rows, contraction tails of 8 to 56
SHAPES = [
    dict(T=1, K=1, E=1, H=8, N=8), dict(T=1, K=2, E=4, H=72, N=40, mask_p=0.0), dict(T=33, K=3, E=5, H=136, N=264),
    dict(T=200, K=2, E=3, H=104, N=520, A=16), dict(T=700, K=2, E=4, H=264, N=136, A=64),
    dict(T=1500, K=1, E=2, H=88, N=272), dict(T=90, K=4, E=1024, H=64, N=48), dict(T=300, K=1, E=1, H=320, N=256),
    dict(T=63, K=1, E=1, H=1000, N=24),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(s[k]) for k in "TKEHN"))
@pytest.mark.parametrize("gather", [False, True])
def test_linear_shapes(shape, gather):
    check(kind="silu", gather=gather, **shape)


@pytest.mark.parametrize("kind", XO.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [40, 900])
def test_linear_activations(kind, gated, T):
    check(T, 2, 4, 136, 168, kind, gated, bias=T == 40, residual=gated, gather=T == 900, seed=5)


@pytest.mark.parametrize("extra", [8, 64])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_rows_in_wider_buffers(extra, gated):
    """Row strides beyond the width, with NaN in the columns beyond."""
    check(150, 2, 3, 72, 88, "gelu", gated, extra=extra, gather=gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,E", [(1200, 6), (150, 6), (2000, 1)])
def test_linear_exact_on_small_integers(gated, T, E):
    """Integers make every sum exact: forward (no activation) and gradients
    equal the rounding of the exact value bit for bit."""
    m = ep()
    H, N, K = 200, 152, 1
    wide = 2 * N if gated else N
    w = W.Workload("i", T=T, H=H, K=K, E=E, mask_p=0.05, seed=3)
    idx, _ = W.make_routing(w)
    L = m.ep_layout(idx.to(DEV), E, expert_alignment=32, expert_row_src=True)
    rows = L.max_expert_rows()
    x, go = W.make_small_ints(w, (rows, H), stream=0), W.make_small_ints(w, (rows, N), stream=1)
    wt, b = W.make_small_ints(w, (E, wide, H), stream=2), W.make_small_ints(w, (E, wide), stream=3)
    res = W.make_small_ints(w, (rows, N), stream=4)
    pre = marked(rows, wide)
    out = m.ep_expert_linear(x.to(DEV), L, wt.to(DEV), bias=b.to(DEV), gated=gated, residual=res.to(DEV), pre=pre)
    who = rows_of(L, False)
    at = np.concatenate([o for _, o in who])
    want, _, z, _ = XO.linear(f64(x), f64(wt), f64(b), "none", gated, f64(res), who)
    if not gated:  # a gated product of two sums may need more than 24 bits
        assert np.array_equal(u16(out)[at], O.bf16_rne(want[at].astype(np.float32)))
    assert np.array_equal(u16(pre)[at], O.bf16_rne(z[at].astype(np.float32)))
    g = go
    if gated:  # gradients of small integers: grad_pre is exact in bf16
        p2 = W.make_small_ints(w, (rows, wide), stream=5)
        gx, gw, gb, gp = m.ep_expert_linear_backward(go.to(DEV), x.to(DEV), L, wt.to(DEV), pre=p2.to(DEV), gated=True,
                                                     bias=True)
        g = torch.cat([go * p2[:, N:], go * p2[:, :N]], 1)
        assert torch.equal(gp.cpu()[at], g[at])
    else:
        gx, gw, gb, _ = m.ep_expert_linear_backward(go.to(DEV), x.to(DEV), L, wt.to(DEV), bias=True)
    (wx, _), (ww, _), (wb, _) = XO.linear_backward(f64(g), f64(x), f64(wt), who)
    assert np.array_equal(u16(gx)[at], O.bf16_rne(wx[at].astype(np.float32)))
    assert np.array_equal(u16(gw), O.bf16_rne(ww.astype(np.float32)))
    assert np.array_equal(u16(gb), O.bf16_rne(wb.astype(np.float32)))


def test_linear_forward_equals_expert_gemm_without_epilogue():
    """The bare product is the grouped GEMM's, bit for bit on exact sums."""
    m = ep()
    w = W.Workload("e", T=800, H=256, K=2, E=5, seed=4)
    idx, _ = W.make_routing(w, device=DEV)
    L = m.ep_layout(idx, w.E)
    x = W.make_small_ints(w, (1600, 256), stream=0, device=DEV)
    wt = W.make_small_ints(w, (5, 384, 256), stream=1, device=DEV)
    assert torch.equal(m.ep_expert_linear(x, L, wt), m.ep_expert_gemm(x, L, wt))


def test_linear_one_expert_has_all_rows():
    """3000 rows of one expert among 40: split over many tiles; the weight
    gradients of the others are zero."""
    idx = torch.full((3000, 1), 17)
    check(3000, 1, 40, 72, 40, "relu", gather=True, idx=idx)


@pytest.mark.parametrize("rows,N", [("even", 520), ("skewed", 520), ("one", 520), ("split", 40)])
def test_linear_weight_gradient_orders(rows, N):
    """32 experts of 160 rows on average, several tiles each: tiles dealt to the
    XCDs by expert where the rows are even, else in runs; and with rows enough
    to be split over blocks."""
    T = 5120 if rows != "split" else 32 * 600
    e = torch.arange(T) % 32
    if rows == "skewed":
        e = torch.where(torch.arange(T) % 3 == 0, torch.full_like(e, 7), e)
    if rows == "one":
        e = torch.full_like(e, 30)
    check(T, 1, 32, 264, N, "relu", gather=rows != "one", idx=e.reshape(T, 1))


@pytest.mark.parametrize("gather", [False, True])
def test_linear_weight_gradient_of_many_rows_is_split(gather):
    """One and two experts with thousands of rows: the rows are split over
    blocks and the parts joined; a second call gives the same bytes."""
    m = ep()
    for E, T in ((1, 5003), (2, 4100)):
        idx = (torch.arange(T) % (E + 1) // 2).reshape(T, 1) if E > 1 else torch.zeros(T, 1, dtype=torch.int64)
        L = m.ep_layout(idx.to(DEV), E, expert_row_src=True)
        assert m.ep_expert_linear_workspace_bytes(L, 64, 72) > 16  # split
        check(T, 1, E, 64, 72, "silu", gather=gather, idx=idx)
        g = torch.Generator().manual_seed(1)
        x, go, w = bf(g, 1, T, 64).to(DEV), bf(g, 1, T, 72).to(DEV), bf(g, 1, E, 72, 64).to(DEV)
        a = m.ep_expert_linear_backward(go, x, L, w, gather=gather, bias=True)
        b = m.ep_expert_linear_backward(go, x, L, w, gather=gather, bias=True)
        assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_linear_nan_and_infinity_stay_in_their_rows():
    """A row of NaN or infinity spoils no other row, forward or in grad_x; an
    expert's weight gradient takes its own rows alone."""
    m = ep()
    T, E, H, N = 100, 3, 72, 40
    idx = (torch.arange(T) % E).reshape(T, 1)
    L = m.ep_layout(idx.to(DEV), E, expert_row_src=True)
    g = torch.Generator().manual_seed(2)
    x, w, go = bf(g, 1, T, H).to(DEV), bf(g, 0.1, E, N, H).to(DEV), bf(g, 1, T, N).to(DEV)
    y = m.ep_expert_linear(x, L, w, gather=True)
    a = m.ep_expert_linear_backward(go, x, L, w, gather=True, bias=True)
    bad = x.clone()
    bad[4] = float("nan")
    bad[7, 3] = float("inf")  # both tokens of expert 1
    gbad = go.clone()
    row = {t: int(L.slot[t, 0]) for t in (4, 7)}
    gbad[row[4], 0] = float("nan")
    y2 = m.ep_expert_linear(bad, L, w, gather=True)
    b = m.ep_expert_linear_backward(gbad, bad, L, w, gather=True, bias=True)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[row[4], row[7]]] = False
    assert torch.equal(y[keep], y2[keep]) and torch.isnan(y2[row[4]]).all()
    assert not torch.isfinite(y2[row[7]]).any()
    keep[row[7]] = True
    assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][row[4]]).all()
    for i in (1, 2):
        assert torch.equal(a[i][[0, 2]], b[i][[0, 2]])
    assert torch.isnan(b[2][1, 0]) and torch.equal(a[2][1, 1:], b[2][1, 1:])


def test_activations_of_large_values():
    """Every finite bf16 has a finite derivative's product and the formula's
    limits: no overflow of an exponential or a cube shows."""
    m = ep()
    z = torch.arange(0, 65536, 1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    n = z.numel() // 8 * 8
    z = z[:n].reshape(-1, 8).contiguous()
    T = z.shape[0]
    L = m.ep_layout(torch.zeros(T, 1, dtype=torch.int64, device=DEV), 1, expert_row_src=True)
    eye = torch.eye(8, dtype=torch.bfloat16, device=DEV)[None]
    one = torch.ones(T, 8, dtype=torch.bfloat16, device=DEV)
    zd = z.to(DEV)
    who = [(np.arange(T), np.arange(T))]
    for kind in XO.ACTS:
        with np.errstate(over="ignore", invalid="ignore"):
            v, d, ev, ed = XO.act(np.clip(f64(z), -1e4, 1e4), kind)  # past 1e4 the limits
        big = np.abs(f64(z)) > 1e4
        out = f64(m.ep_expert_linear(zd, L, eye, activation=act_id(kind)))
        want = np.where(big, (f64(z) if kind == "none" else np.maximum(f64(z), 0)), v)
        tol = 2.0**-8 * np.abs(want) + 2 * ev + 2.0**-120
        assert (np.abs(out - want) <= tol).all(), kind
        if kind == "none":
            continue
        gp = f64(m.ep_expert_linear_backward(one, zd, L, eye, pre=zd, activation=act_id(kind), needs=(False, False))[3])
        want = np.where(big, (f64(z) > 0).astype(float), d)
        assert (np.abs(gp - want) <= 2.0**-8 * np.abs(want) + 2 * ed + 2.0**-120).all(), kind


def test_linear_in_place_and_partial_gradients():
    m = ep()
    w = W.Workload("p", T=130, H=64, K=2, E=4, mask_p=0.1, seed=8)
    idx, _ = W.make_routing(w, device=DEV)
    L = m.ep_layout(idx, 4, expert_row_src=True)
    g = torch.Generator().manual_seed(3)
    x, wt, res = bf(g, 1, 130, 64).to(DEV), bf(g, 0.1, 4, 96, 64).to(DEV), bf(g, 1, 260, 48).to(DEV)
    pre = marked(260, 96)
    kw = dict(activation=m.EP_ACT_SILU, gated=True, gather=True)
    want = m.ep_expert_linear(x, L, wt, residual=res, out=res.clone(), pre=pre, **kw)
    out = res.clone()
    assert m.ep_expert_linear(x, L, wt, residual=out, out=out, **kw) is out and torch.equal(out, want)
    # grad_pre over pre; one gradient at a time
    go = bf(g, 1, 260, 48).to(DEV)
    full = m.ep_expert_linear_backward(go, x, L, wt, pre=pre, bias=True, **kw)
    live = L.num_rows()
    p2 = pre.clone()
    only_x = m.ep_expert_linear_backward(go, x, L, wt, pre=p2, grad_pre=p2, needs=(True, False), **kw)
    assert only_x[1] is None and only_x[2] is None and only_x[3] is p2
    assert torch.equal(only_x[0][:live], full[0][:live]) and torch.equal(p2[:live], full[3][:live])
    only_w = m.ep_expert_linear_backward(go, x, L, wt, pre=pre, needs=(False, True), **kw)
    assert only_w[0] is None and only_w[2] is None and torch.equal(only_w[1], full[1])


@pytest.mark.parametrize("T,K,E,H,N,gather", [
    (40, 2, 8, 264, 120, False),     # a few rows an expert
    (300, 2, 8, 1032, 520, True),    # about 70
    (1100, 1, 4, 520, 1288, False),  # about 270
    (4000, 2, 33, 264, 520, True),   # about 240, many experts
    (3000, 1, 1, 264, 264, False),   # one expert, rows split
])
def test_linear_gradients_together_equal_each_alone(T, K, E, H, N, gather):
    print(f"together T={T} K={K} E={E} H={H} N={N} gather={gather}", flush=True)
    m = ep()
    idx, _ = W.make_routing(W.Workload("x", T=T, H=H, K=K, E=E, mask_p=0.1, seed=T + 1))
    L = m.ep_layout(idx.to(DEV), E, expert_row_src=True)
    rows = L.max_expert_rows()
    g = torch.Generator().manual_seed(T)
    x, go = bf(g, 1.0, T if gather else rows, H).to(DEV), bf(g, 1.0, rows, N).to(DEV)
    w = bf(g, H**-0.5, E, N, H).to(DEV)
    kw = dict(gather=gather)
    gx, gw, gb, _ = m.ep_expert_linear_backward(go, x, L, w, bias=True, grad_x=marked(rows, H), **kw)
    ax, none, _, _ = m.ep_expert_linear_backward(go, x, L, w, grad_x=marked(rows, H), needs=(True, False), **kw)
    assert none is None
    none, aw, ab, _ = m.ep_expert_linear_backward(go, x, L, w, bias=True, needs=(False, True), **kw)
    assert none is None
    torch.cuda.synchronize()
    assert np.array_equal(u16(gx), u16(ax))
    assert np.array_equal(u16(gw), u16(aw)) and np.array_equal(u16(gb), u16(ab))


def test_linear_stale_empty_and_refused():
    m = ep()
    w = W.Workload("s", T=20, H=64, K=1, E=2, seed=9)
    idx, _ = W.make_routing(w, device=DEV)
    L = m.ep_layout(idx, 2, expert_row_src=True)
    x = torch.ones(20, 64, dtype=torch.bfloat16, device=DEV)
    wt = torch.ones(2, 32, 64, dtype=torch.bfloat16, device=DEV)
    handle = L.handle()
    old = L.generation
    m.ep_layout(idx, 2, expert_row_src=True, out=L)
    with pytest.raises(m.StaleLayoutError if hasattr(m, "StaleLayoutError") else RuntimeError):
        m.ep_expert_linear(x, handle, wt)
    L.generation = old
    out, gx, gw, gb = marked(20, 32), marked(20, 64), marked(2 * 32, 64).reshape(2, 32, 64), marked(2, 32)
    m.ep_expert_linear(x, L, wt, out=out)
    m.ep_expert_linear_backward(out, x, L, wt, grad_x=gx, grad_w=gw, grad_bias=gb)
    torch.cuda.synchronize()
    assert all((u16(t) == 0xFFFF).all() for t in (out, gx, gw, gb)) and L.stale_call_seen()
    # no token: the weights' gradients are zero
    L0 = m.ep_layout(idx[:0], 2, expert_row_src=True)
    assert m.ep_expert_linear(x[:0], L0, wt).shape == (0, 32)
    gx, gw, gb, _ = m.ep_expert_linear_backward(out[:0], x[:0], L0, wt, bias=True)
    assert gx.shape == (0, 64) and (gw == 0).all() and (gb == 0).all()
    with pytest.raises(m.EPError):
        m.ep_expert_linear(x, L, wt, out=x)


def test_linear_offsets_past_32_bits():
    """Rows and weights whose byte offsets pass 2^32: the last rows and the
    last expert as in a small call of their own."""
    m = ep()
    T, H, N = 150_000, 16_384, 64  # x: 4.9 GB
    E = 3
    idx = torch.full((T, 1), 0, dtype=torch.int64, device=DEV)
    idx[-50:] = 2
    L = m.ep_layout(idx, E, expert_row_src=True)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    x[-50:] = torch.randn(50, H, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(E, N, H, generator=g, device=DEV) * H**-0.5).to(torch.bfloat16)
    go = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    L1 = m.ep_layout(idx[-50:] - 2, 1, expert_row_src=True)
    for gather in (False, True):
        y = m.ep_expert_linear(x, L, w, gather=gather)
        y1 = m.ep_expert_linear(x[-50:].contiguous(), L1, w[2:].contiguous())
        # the 50 rows may fall into tiles of another height: same operands, same order
        assert torch.equal(y[-50:], y1)
        gx, gw, gb, _ = m.ep_expert_linear_backward(go, x, L, w, gather=gather, bias=True)
        gx1, gw1, gb1, _ = m.ep_expert_linear_backward(go[-50:].contiguous(), x[-50:].contiguous(), L1,
                                                       w[2:].contiguous(), bias=True)
        assert torch.equal(gx[-50:], gx1) and torch.equal(gb[2], gb1[0])
        # the many rows are split over blocks, the 50 are not: each sum is within
        # half a bf16 step and 50 fp32 additions in any order of the exact one
        g64, x64 = go[-50:].double().cpu(), x[-50:].double().cpu()
        exact, size = g64.T @ x64, g64.abs().T @ x64.abs()
        for got in (gw[2], gw1[0]):
            assert ((got.double().cpu() - exact).abs() <= 2.0**-8 * exact.abs() + 100 * XO.U32 * size).all()
        assert (gw[0] == 0).all() and (gw[1] == 0).all()
        del y, gx, gw


def test_linear_many_weights_past_32_bits():
    """Expert weights of 4.8 GB: the last expert's layer and gradients."""
    m = ep()
    E, H, N, T = 300, 4096, 2048, 600
    w = torch.zeros(E, N, H, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    w[-1] = (torch.randn(N, H, generator=g, device=DEV) * H**-0.5).to(torch.bfloat16)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    go = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    idx = (torch.arange(T, device=DEV) % E).reshape(T, 1)
    L = m.ep_layout(idx, E, expert_row_src=True)
    L1 = m.ep_layout(torch.zeros(2, 1, dtype=torch.int64, device=DEV), 1)
    at = L.slot.reshape(-1)[[E - 1, 2 * E - 1]].long()
    xr = m.ep_dispatch(x, L)
    y, y1 = m.ep_expert_linear(xr, L, w), m.ep_expert_linear(xr[at].contiguous(), L1, w[-1:].contiguous())
    assert torch.equal(y[at], y1)
    a = m.ep_expert_linear_backward(go, xr, L, w)
    b = m.ep_expert_linear_backward(go[at].contiguous(), xr[at].contiguous(), L1, w[-1:].contiguous())
    assert torch.equal(a[0][at], b[0]) and torch.equal(a[1][-1], b[1][0])


def test_linear_captured_in_a_graph_and_on_another_stream():
    """Forward and gradients captured once; replays with new inputs equal eager
    calls, with eager work between them; a side stream gives the same."""
    m = ep()
    w = W.Workload("gr", T=2100, H=72, K=1, E=2, mask_p=0.1, seed=12)
    idx, _ = W.make_routing(w, device=DEV)
    L = m.ep_layout(idx, 2, expert_row_src=True)
    g = torch.Generator().manual_seed(6)
    x, wt, b = bf(g, 1, 2100, 72).to(DEV), bf(g, 0.1, 2, 80, 72).to(DEV), bf(g, 1, 2, 80).to(DEV)
    go = bf(g, 1, 2100, 40).to(DEV)
    kw = dict(activation=m.EP_ACT_GELU, gated=True, gather=True)
    ws = torch.empty(m.ep_expert_linear_workspace_bytes(L, 72, 40, gated=True), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 16  # the rows are split

    def step(bufs):
        out, pre, gx, gw, gb, gp = bufs
        m.ep_expert_linear(x, L, wt, bias=b, out=out, pre=pre, **kw)
        m.ep_expert_linear_backward(go, x, L, wt, pre=pre, grad_x=gx, grad_w=gw, grad_bias=gb, grad_pre=gp,
                                    workspace=ws, **kw)

    def fresh():
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        return z(2100, 40), z(2100, 80), z(2100, 72), z(2, 80, 72), z(2, 80), z(2100, 80)

    bufs = fresh()
    step(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs)
    for k in range(3):
        x.copy_(bf(g, 1, 2100, 72))
        go.copy_(bf(g, 1, 2100, 40))
        want = fresh()
        step(want)
        torch.cuda.synchronize()
        for t in bufs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(bufs, want)), k
    side = torch.cuda.Stream()
    other = fresh()
    with torch.cuda.stream(side):
        step(other)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, want))
