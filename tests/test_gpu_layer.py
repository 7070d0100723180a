"""GPU tests of the combine's gradient (grad_y bit for bit, grad_weights within
a derived bound) and of the layer operators run together, as a step that
trains a router and adapters on frozen experts."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import ep_oracle as O
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


def f64(t):
    return t.detach().cpu().double().numpy()


def u16(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def _check_combine(go, y, L, w, y_rows_seen=None):
    m = ep()
    gy = torch.full(y.shape, -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    gw = torch.full(w.shape, 9.0, device=DEV)
    m.ep_combine_backward(go, y, L, w, grad_y=gy, grad_weights=gw)
    torch.cuda.synchronize()
    want_y, want_w, bound = LO.combine_backward(f64(go), f64(y), L.slot.cpu().numpy(), w.cpu().numpy())
    wrote = ~np.isnan(want_y)
    got = u16(gy)
    assert np.array_equal(got[wrote], O.bf16_rne(want_y[wrote]))
    assert (got[~wrote] == 0xFFFF).all()  # rows of no selection: left as they were
    err = np.abs(f64(gw) - want_w)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("T,H,K,E,A", [
    (1, 1, 1, 1, 0), (1, 7168, 8, 64, 0), (5, 2, 3, 8, 0), (9, 3, 2, 4, 0), (128, 256, 2, 16, 0), (33, 520, 5, 16, 4),
    (17, 1030, 8, 32, 0), (6, 2049, 4, 8, 0), (11, 4100, 13, 64, 16), (4, 640, 32, 64, 0), (70, 512, 1, 4, 0),
])
def test_combine_backward(T, H, K, E, A):
    print(f"combine backward T={T} H={H} K={K} E={E} A={A}", flush=True)
    w = W.Workload("cb", T=T, H=H, K=K, E=E, mask_p=0.15, seed=T + H)
    idx, wt = W.make_routing(w)
    L = ep().ep_layout(idx.to(DEV), E, expert_alignment=A)
    _check_combine(W.make_x(w.replace(seed=3)).to(DEV), W.make_y(w, L.max_expert_rows()).to(DEV), L, wt.to(DEV))


def test_combine_backward_full_size_sampled():
    """8192 tokens x 7168, top-8 of 256: grad_y of every row against torch's
    fp32 product rounded once, grad_weights of 64 tokens against the oracle."""
    w = W.by_name("pages")
    idx, wt = W.make_routing(w, device=DEV)
    L = ep().ep_layout(idx, w.E)
    y, go = W.make_y(w, device=DEV), W.make_x(w, device=DEV)
    gy, gw = ep().ep_combine_backward(go, y, L, wt)
    slot = L.slot.long()
    for k in range(w.K):
        want = (wt[:, k:k + 1] * go.float()).to(torch.bfloat16)
        assert torch.equal(gy[slot[:, k]], want)
    t = torch.arange(0, w.T, 128, device=DEV)
    rows = slot[t].reshape(-1)
    small = torch.arange(rows.numel()).reshape(len(t), w.K)
    _, want_w, bound = LO.combine_backward(f64(go[t]), f64(y[rows]), small.numpy(), wt[t].cpu().numpy())
    assert (np.abs(f64(gw[t]) - want_w) <= bound).all()


def test_combine_backward_offsets_past_32_bits():
    """80,000 expert rows x 32,768 (5.2 GB): the last tokens as in a call on
    rows of their own."""
    m = ep()
    T, H = 80_000, 32_768
    idx = torch.zeros(T, 1, dtype=torch.int64, device=DEV)
    L = m.ep_layout(idx, 1)
    wt = torch.full((T, 1), 0.5, device=DEV)
    go = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    w = W.Workload("cb", T=40, H=H, K=1, E=1, seed=2)
    go[-40:], y[-40:] = W.make_x(w, device=DEV), W.make_y(w, device=DEV)
    gy, gw = m.ep_combine_backward(go, y, L, wt)
    L1 = m.ep_layout(idx[-40:], 1)
    one = m.ep_combine_backward(go[-40:].clone(), y[-40:].clone(), L1, wt[-40:])
    assert torch.equal(gy[-40:], one[0]) and torch.equal(gw[-40:], one[1])
    assert (gy[:-40] == 0).all() and (gw[:-40] == 0).all()


def test_combine_backward_masked_oob_and_misaligned():
    m = ep()
    w = W.Workload("cb", T=50, H=264, K=4, E=8, seed=5)
    idx, wt = W.make_routing(w)
    idx[3] = -1
    L = m.ep_layout(idx.to(DEV), w.E)
    rows = L.max_expert_rows()
    go, y = W.make_x(w).to(DEV), W.make_y(w).to(DEV)
    # bases at 2-byte alignment
    flat = torch.zeros(rows * w.H + 1, dtype=torch.bfloat16, device=DEV)
    flat[1:] = y.reshape(-1)
    _check_combine(go, flat[1:].reshape(rows, w.H), L, wt.to(DEV))
    # fewer y rows than the layout has: the rest is skipped and reported
    assert L.status_word(m.EP_STATUS_COMBINE_OOB) == 0
    _check_combine(go, y[:100].contiguous(), L, wt.to(DEV))
    assert L.status_word(m.EP_STATUS_COMBINE_OOB) == 1
    # infinities in rows of no selection and in a masked token have no effect
    go2 = go.clone()
    go2[3] = float("nan")
    a, b = m.ep_combine_backward(go, y, L, wt.to(DEV)), m.ep_combine_backward(go2, y, L, wt.to(DEV))
    live = (L.slot.reshape(-1)[L.slot.reshape(-1) >= 0]).long()
    assert torch.equal(a[0][live], b[0][live]) and torch.equal(a[1], b[1])
    # a stale struct writes nothing
    old = L.generation
    m.ep_layout(idx.to(DEV), w.E, out=L)
    L.generation = old
    gy, gw = torch.full_like(y, 5.0), torch.full_like(wt, 5.0).to(DEV)
    m.ep_combine_backward(go, y, L, wt.to(DEV), grad_y=gy, grad_weights=gw)
    assert (gy == 5).all() and (gw == 5).all() and L.stale_call_seen()
    with pytest.raises(m.EPError):
        m.ep_combine_backward(go, y, L, wt.to(DEV), grad_y=y)
    # T = 0
    L0 = m.ep_layout(idx[:0].to(DEV), w.E)
    gy, gw = m.ep_combine_backward(go[:0], y[:0], L0, wt[:0].to(DEV))
    assert gy.shape == (0, w.H) and gw.shape == (0, w.K)


def test_combine_backward_is_the_derivative_of_combine():
    """<grad_out, combine(y + d) - combine(y)> against <grad_y, d>: both sides
    from the kernels, to the accuracy of bf16 outputs."""
    m = ep()
    w = W.Workload("cb", T=64, H=256, K=4, E=8, mask_p=0.1, seed=6)
    idx, wt = (t.to(DEV) for t in W.make_routing(w))
    L = m.ep_layout(idx, w.E)
    y, d, go = (W.make_small_ints(w, (256, w.H), stream=i, device=DEV) for i in range(3))
    go = go[: w.T].contiguous()
    wt = torch.full_like(wt, 0.5)  # exact in bf16 and in every sum
    gy, gw = m.ep_combine_backward(go, y, L, wt)
    live = L.slot.reshape(-1)[L.slot.reshape(-1) >= 0].long()
    diff = m.ep_combine(y + d, L, wt).double() - m.ep_combine(y, L, wt).double()
    assert float((go.double() * diff).sum()) == float((gy[live].double() * d[live].double()).sum())
    # in the weights it is linear too: one weight at a time
    ones = torch.zeros_like(wt)
    ones[:, 2] = 1.0
    one = m.ep_combine(y, L, ones).double()
    assert torch.equal((go.double() * one).sum(1), gw[:, 2].double())


def test_training_step_of_router_and_adapters():
    """route -> layout -> dispatch -> grouped GEMM beside adapters -> combine,
    and back, against the same layer in float64 torch autograd.

    The kernels round to bf16 four times on the way of a gradient (the GEMM's
    output, the adapters' output, grad_y, the result), each by at most 2^-8 of
    the value's size and independently, so a gradient's 2-norm error stays
    below 4 * 2^-8; the selections are equal."""
    m = ep()
    T, H, N, E, K, R = 192, 128, 128, 16, 4, 16
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rnd(T, H).to(torch.bfloat16)
    logits = (rnd(T, E) * 1.5)
    bias = (rnd(E) * 40).round() * 1e-3
    wts = (rnd(E, N, H) * H**-0.5).to(torch.bfloat16)
    a, b = (rnd(E, R, H) * H**-0.5).to(torch.bfloat16), (rnd(E, N, R) * R**-0.5).to(torch.bfloat16)
    scales = torch.rand(E, generator=g) + 0.5
    go = rnd(T, N).to(torch.bfloat16)
    dx, dl, db, dw, da, dbb, ds, dgo = (t.to(DEV) for t in (x, logits, bias, wts, a, b, scales, go))
    kw = dict(score=m.EP_SCORE_SIGMOID, renormalize=True, scale=2.0)

    # forward
    idx, w = m.ep_route(dl, K, bias=db, num_groups=4, topk_groups=2, group_top=2, **kw)
    L = m.ep_layout(idx, E, expert_row_src=True)
    xr = m.ep_dispatch(dx, L)
    y = m.ep_expert_gemm(xr, L, dw)
    m.ep_lora(xr, L, da, dbb, base=y, scales=ds, out=y)
    out = m.ep_combine(y, L, w)
    # the adapters beside the GEMM whose dispatch is folded into its loads: the same rows
    y2 = m.ep_expert_gemm(dx, L, dw, gather=True)
    m.ep_lora(dx, L, da, dbb, base=y2, scales=ds, out=y2, gather=True)
    assert torch.equal(y, y2)
    # backward
    gy, gw = m.ep_combine_backward(dgo, y, L, w)
    gl = m.ep_route_backward(gw, dl, idx, **kw)
    gxr = m.ep_expert_gemm(gy, L, dw.transpose(1, 2).contiguous())
    gxr, ga, gb = m.ep_lora_backward(gy, xr, L, da, dbb, scales=ds, grad_base=gxr, grad_x=gxr)
    gx = m.ep_combine(gxr, L, torch.ones_like(w))
    torch.cuda.synchronize()

    # the same in float64
    rx, rl, ra, rb = (t.double().requires_grad_() for t in (x, logits, a, b))
    want_i, _ = LO.route(f64(logits), K, "sigmoid", f64(bias), 4, 2, 2, True, 2.0)
    assert np.array_equal(idx.cpu().numpy(), want_i)
    ri = torch.from_numpy(want_i)
    p = torch.sigmoid(torch.gather(rl, 1, ri))
    rw = 2.0 * p / p.sum(1, keepdim=True)
    wd = wts.double()
    ro = torch.zeros(T, N, dtype=torch.float64)
    for k in range(K):
        e = ri[:, k]
        base = (wd[e] @ rx[:, :, None])[:, :, 0]
        low = scales.double()[e, None] * (rb[e] @ (ra[e] @ rx[:, :, None]))[:, :, 0]
        ro = ro + rw[:, k:k + 1] * (base + low)
    (ro * go.double()).sum().backward()

    def close(got, want, n):
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= n * 2.0**-8, rel

    close(out, ro.detach(), 3)
    close(gx, rx.grad, 4)
    close(ga, ra.grad, 4)
    close(gb, rb.grad, 4)
    close(gl, rl.grad, 4)
