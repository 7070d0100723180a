"""GPU parity of the low-rank adapters and their gradients against the float64
oracle, within bounds derived there; bit-exact on small integers."""
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


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """Inputs of one call: ids [T, K] over E adapters, sizes, row modes."""

    def __init__(self, ids, E, H, N, R, gather=False, scatter=False, A=0, seed=0, ints=False, scaled=True, pad=0):
        m = ep()
        g = torch.Generator().manual_seed(seed)
        self.ids, self.E, self.H, self.N, self.R, self.gather, self.scatter = ids, E, H, N, R, gather, scatter
        self.L = m.ep_layout(ids.to(DEV), E, expert_alignment=A, expert_row_src=True)
        rows, T = self.L.max_expert_rows(), ids.shape[0]
        xr, orows = T if gather else rows, T if scatter else rows

        def make(*shape, std=1.0):
            if ints:
                return torch.randint(-2, 3, shape, generator=g).to(torch.bfloat16)
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)

        self.x, self.go = make(xr, H + pad), make(orows, N + pad)
        self.a, self.b = make(E, R, H, std=H**-0.5), make(E, N, R, std=R**-0.5)
        self.base, self.gbase = make(orows, N + pad), make(orows, H + pad)
        self.scales = torch.rand(E, generator=g) + 0.5 if scaled else None
        if ints and scaled:
            self.scales = torch.full((E,), 0.5)
        # rows of x and of out, expert by expert, from the layout's own definition
        counts, offsets = self.L.counts.cpu().numpy(), self.L.offsets.cpu().numpy()
        src = self.L.expert_row_src.cpu().numpy()
        self.rows_of = []
        self.selected = np.zeros(orows, bool)
        for e in range(E):
            r = np.arange(offsets[e], offsets[e] + counts[e])
            xi, oi = (src[r] if gather else r), (src[r] if scatter else r)
            self.rows_of.append((xi, oi))
            self.selected[oi] = True
        # what belongs to no selection must not be read: poison it
        xsel = np.zeros(xr, bool)
        for xi, _ in self.rows_of:
            xsel[xi] = True
        self.x[~torch.from_numpy(xsel)] = float("nan")
        self.go[~torch.from_numpy(self.selected)] = float("inf")
        if pad:
            self.x[:, H:] = float("nan")
            self.go[:, N:] = float("nan")
        self.dev = {k: None if v is None else v.to(DEV) for k, v in
                    dict(x=self.x, go=self.go, a=self.a, b=self.b, base=self.base, gbase=self.gbase,
                         scales=self.scales).items()}
        self.s64 = np.ones(E) if self.scales is None else f64(self.scales)
        self.kw = dict(scales=self.dev["scales"], gather=gather, scatter=scatter)

    def forward(self, base=True, inplace=False):
        m, d = ep(), self.dev
        poison = torch.full(self.base.shape, -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        bt = d["base"].clone() if base else None
        out = bt if inplace else poison.clone()
        got = m.ep_lora(d["x"], self.L, d["a"], d["b"], base=bt, out=out, **self.kw)
        assert got is out
        b64 = f64(self.base)[:, : self.N] if base else np.zeros((len(self.base), self.N))
        want, bound = LO.lora(f64(self.x)[:, : self.H], f64(self.a), f64(self.b), self.s64, b64, self.rows_of)
        got64 = f64(got)[:, : self.N]
        err = np.abs(got64 - want)
        sel = self.selected
        assert (err[sel] <= bound[sel]).all(), (err[sel] - bound[sel]).max()
        rest = torch.from_numpy(~sel)
        untouched = self.base.view(torch.int16) if inplace else poison.cpu().view(torch.int16)
        mine = got.cpu().view(torch.int16)
        if self.scatter and not inplace:
            assert np.array_equal(got64[~sel], b64[~sel])
        else:
            assert torch.equal(mine[rest], untouched[rest])
        assert torch.equal(mine[:, self.N:], untouched[:, self.N:])  # past the width: never written
        return got, want

    def backward(self, base=False):
        m, d = ep(), self.dev
        orows = len(self.base)
        gx = torch.full((orows, self.gbase.shape[1]), -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        ga = torch.full(self.a.shape, -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        gb = torch.full(self.b.shape, -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        m.ep_lora_backward(d["go"], d["x"], self.L, d["a"], d["b"], grad_base=d["gbase"] if base else None, grad_x=gx,
                           grad_a=ga, grad_b=gb, **self.kw)
        b64 = f64(self.gbase)[:, : self.H] if base else np.zeros((orows, self.H))
        want = LO.lora_backward(f64(self.go)[:, : self.N], f64(self.x)[:, : self.H], f64(self.a), f64(self.b), self.s64,
                                b64, self.rows_of)
        sel = self.selected
        for name, got, (w, bound) in zip(("grad_x", "grad_a", "grad_b"), (gx, ga, gb), want):
            v = f64(got)
            if name == "grad_x":
                if self.scatter:
                    assert np.array_equal(v[~sel][:, : self.H], b64[~sel])
                else:
                    assert (got.cpu().view(torch.int16)[torch.from_numpy(~sel)] == -1).all()
                v, w, bound = v[sel][:, : self.H], w[sel], bound[sel]
            err = np.abs(v - w)
            assert (err <= bound).all(), (name, (err - bound).max())
        return gx, ga, gb, want


def _ids(T, K, E, seed, none=0.1, uneven=True):
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) ** (3 if uneven else 0) + 1e-3
    ids = torch.multinomial(p.expand(T, E), K, generator=g)
    return torch.where(torch.rand(T, K, generator=g) < none, -1, ids)


# T, K, E, H, N, R, gather, scatter, alignment, width past H and N
CASES = [
    (1, 1, 1, 8, 8, 8, True, True, 0, 0),
    (1, 1, 48, 4096, 1024, 16, True, True, 0, 0),
    (5, 1, 3, 72, 136, 24, True, True, 0, 8),
    (61, 1, 48, 520, 264, 16, True, True, 0, 0),
    (200, 1, 4, 256, 640, 32, True, True, 0, 0),
    (333, 1, 2, 136, 128, 64, True, True, 16, 0),
    (130, 1, 2, 264, 72, 128, True, True, 0, 16),
    (150, 1, 2, 64, 520, 104, False, True, 0, 0),
    (90, 3, 8, 128, 256, 8, False, False, 0, 0),
    (256, 4, 16, 320, 192, 40, True, False, 64, 8),
    (300, 2, 3, 1032, 1032, 16, False, False, 32, 0),
    (40, 2, 1024, 64, 64, 16, True, False, 0, 0),
    (700, 1, 1000, 64, 128, 8, True, True, 0, 0),
]


# 2048 rows and more, 32 and more per expert: tiles of 32 and 64 rows, result
# tiles of 64 and 128 rows, experts of several weight-gradient chunks
LARGE = [
    (2100, 1, 8, 136, 264, 16, True, True, 0, 0),
    (2100, 1, 40, 72, 520, 32, True, True, 0, 8),
    (4200, 1, 9, 200, 136, 8, True, True, 0, 0),
    (4200, 1, 5, 1096, 1032, 24, True, True, 0, 0),
    (2200, 2, 16, 128, 640, 32, False, False, 64, 0),
    (2200, 2, 30, 328, 512, 64, True, False, 0, 16),
    (4500, 1, 6, 264, 200, 128, True, True, 0, 0),
    (4500, 1, 20, 64, 1160, 112, True, True, 0, 0),
    (1500, 4, 5, 520, 72, 48, False, False, 0, 0),
]
CASES = CASES + LARGE


@pytest.mark.parametrize("T,K,E,H,N,R,gather,scatter,A,pad", CASES)
def test_lora(T, K, E, H, N, R, gather, scatter, A, pad):
    print(f"lora T={T} K={K} E={E} H={H} N={N} R={R} gather={gather} scatter={scatter} A={A} pad={pad}", flush=True)
    c = Case(_ids(T, K, E, T + R), E, H, N, R, gather, scatter, A, seed=T, pad=pad)
    c.forward()
    c.forward(inplace=True)
    c.forward(base=False)


@pytest.mark.parametrize("T,K,E,H,N,R,gather,scatter,A,pad", CASES)
def test_lora_backward(T, K, E, H, N, R, gather, scatter, A, pad):
    print(f"lora backward T={T} K={K} E={E} H={H} N={N} R={R} gather={gather} scatter={scatter} A={A}", flush=True)
    c = Case(_ids(T, K, E, T + R), E, H, N, R, gather, scatter, A, seed=T, pad=pad, scaled=T % 2 == 0)
    c.backward()
    c.backward(base=True)


@pytest.mark.parametrize("T,K,E,H,N,R,scatter", [(33_000, 1, 7, 1024, 264, 16, True), (17_000, 2, 70, 1000, 520, 40, False),
                                                 (33_000, 1, 3, 1016, 72, 72, True)])
def test_lora_more_rows_than_caches_keep(T, K, E, H, N, R, scatter):
    """64 MiB of rows and more, loaded another way; more tokens without an
    adapter than the blocks that copy them take at once."""
    assert T * K * H * 2 >= 64 << 20 or T * K * (H + N) * 2 >= 64 << 20
    c = Case(_ids(T, K, E, T + R, none=0.4), E, H, N, R, True, scatter, seed=R)
    c.forward()
    c.forward(inplace=True)
    c.backward(base=True)


@pytest.mark.parametrize("gather,scatter,K,T", [(True, True, 1, 150), (False, False, 2, 150), (True, True, 1, 2500),
                                                (True, False, 2, 2500)])
@pytest.mark.parametrize("R", [8, 16, 32, 72, 128])
def test_lora_exact_on_small_integers(R, gather, scatter, K, T):
    """Integers in [-2, 2] and a scale of one half: u and v have at most 16
    significand bits (|u| <= 4 H = 2^13 and |v| <= 4 N < 2^13) and every fp32
    sum is exact (below 2^24 in units of one half), so each result is the
    bf16 rounding of the exact value: any misplaced row, column or rank shows."""
    H, N = 2048, 904
    c = Case(_ids(T, K, 5, R), 5, H, N, R, gather, scatter, seed=R, ints=True)
    got, want = c.forward()
    sel = torch.from_numpy(c.selected)
    assert torch.equal(got.cpu()[sel], torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)[sel])
    gx, ga, gb, w = c.backward()
    for name, g, (v, _) in zip("xab", (gx, ga, gb), w):
        v = torch.from_numpy(v)
        assert v.abs().max() < 2**23
        g, v = (g.cpu()[sel], v[sel]) if name == "x" else (g.cpu(), v)
        assert torch.equal(g, v.to(torch.float32).to(torch.bfloat16)), name


def test_lora_one_adapter_with_most_rows():
    """A chunk count above one for one expert, exactly one for others, none for
    the rest: partial gradients joined, written directly, and zeroed."""
    ids = torch.full((1000, 1), 3)
    ids[:64] = 1
    ids[64:128] = -1
    ids[128] = 6
    c = Case(ids, 8, 136, 264, 16, True, True, seed=2)
    c.forward()
    gx, ga, gb, _ = c.backward(base=True)
    for e in (0, 2, 4, 5, 7):
        assert (ga[e] == 0).all() and (gb[e] == 0).all()


def test_lora_no_selection_at_all():
    ids = torch.full((20, 1), -1)
    c = Case(ids, 4, 64, 64, 8, True, True)
    c.forward()
    c.forward(base=False)
    gx, ga, gb, _ = c.backward()
    assert (gx == 0).all() and (ga == 0).all() and (gb == 0).all()
    m = ep()
    L = m.ep_layout(ids[:0].to(DEV), 4, expert_row_src=True)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    out = m.ep_lora(x, L, c.dev["a"], c.dev["b"], gather=True, scatter=True)
    assert out.shape == (0, 64)
    got = m.ep_lora_backward(out, x, L, c.dev["a"], c.dev["b"], gather=True, scatter=True,
                             grad_a=torch.ones_like(c.dev["a"]), grad_b=torch.ones_like(c.dev["b"]))
    assert got[0].shape == (0, 64) and (got[1] == 0).all() and (got[2] == 0).all()


def test_lora_infinities_stay_in_their_rows():
    """An infinite or NaN element makes its own row infinite or NaN and no
    other; u too large for bf16 becomes infinite, not NaN."""
    c = Case(torch.zeros(40, 1, dtype=torch.int64), 1, 64, 64, 16, True, True, seed=4, scaled=False)
    x, clean = c.dev["x"].clone(), c.dev["x"].clone()
    x[7, 3], x[20, 5] = float("inf"), float("nan")
    a, b = c.dev["a"].abs() + 0.01, c.dev["b"].abs() + 0.01
    m = ep()
    got = m.ep_lora(x, c.L, a, b, gather=True, scatter=True)
    want = m.ep_lora(clean, c.L, a, b, gather=True, scatter=True)
    assert torch.isposinf(got[7]).all() and torch.isnan(got[20]).all()
    keep = torch.ones(40, dtype=torch.bool)
    keep[[7, 20]] = False
    assert torch.equal(got[keep], want[keep])
    x[7], x[20] = 3e38, 0.0
    got = m.ep_lora(x, c.L, a, b, gather=True, scatter=True)
    assert torch.isposinf(got[7]).all() and (got[20] == 0).all()


def test_lora_offsets_past_32_bits():
    """70,000 token rows 32,768 elements apart (4.6 GB): the last requests as
    in a call on compact rows."""
    m = ep()
    T, E, H, N, R, W = 70_000, 3, 128, 136, 16, 32_768
    ids = torch.full((T, 1), -1, device=DEV)
    ids[-500:] = _ids(500, 1, E, 5).to(DEV)
    small = Case(ids[-500:].cpu(), E, H, N, R, True, True, seed=9)
    d = small.dev
    go, xs = d["go"].nan_to_num(0.0, posinf=0.0), d["x"].nan_to_num(0.0)
    L = m.ep_layout(ids, E, expert_row_src=True)
    big = torch.zeros(T, W, dtype=torch.bfloat16, device=DEV)
    big[-500:, :H] = xs
    base = torch.zeros(T, W, dtype=torch.bfloat16, device=DEV)
    base[-500:, :N] = d["base"]
    m.ep_lora(big, L, d["a"], d["b"], base=base, out=base, **small.kw)
    want = m.ep_lora(xs, small.L, d["a"], d["b"], base=d["base"], **small.kw)

    def close(got, want):
        # the two calls may split a contraction differently: each result is
        # within half a bf16 step of nearly the same value, one step in all
        got, want = got.double(), want.double()
        return ((got - want).abs() <= 2 * LO.UBF * want.abs() + 1e-3).all()

    assert close(base[-500:, :N], want) and (base[:-500] == 0).all()
    base[-500:, :N] = go
    gx, ga, gb = m.ep_lora_backward(base, big, L, d["a"], d["b"], **small.kw)
    want = m.ep_lora_backward(go, xs, small.L, d["a"], d["b"], **small.kw)
    assert close(gx[-500:], want[0]) and close(ga, want[1]) and close(gb, want[2]) and (gx[:-500] == 0).all()


def test_lora_refuses_and_stale():
    m = ep()
    c = Case(_ids(20, 2, 4, 1), 4, 64, 64, 8)
    d = c.dev
    with pytest.raises(ValueError, match="one selection"):
        m.ep_lora(d["x"], c.L, d["a"], d["b"], scatter=True)
    with pytest.raises(m.EPError):
        m.ep_lora(d["x"], c.L, d["a"], d["b"], out=d["x"])
    with pytest.raises(m.EPError):
        m.ep_lora(d["x"], c.L, d["a"], d["b"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    bare = m.ep_layout(c.ids.to(DEV), 4)
    with pytest.raises(ValueError, match="expert_row_src"):
        m.ep_lora(d["x"], bare, d["a"], d["b"], gather=True)
    # on the device: a struct from before the last layout writes nothing
    old = c.L.generation
    m.ep_layout(c.ids.to(DEV), 4, out=c.L)
    c.L.generation = old
    out = torch.full((c.L.max_expert_rows(), 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ga = torch.full_like(d["a"], 7.0)
    m.ep_lora(d["x"], c.L, d["a"], d["b"], out=out)
    m.ep_lora_backward(d["go"], d["x"], c.L, d["a"], d["b"], grad_x=out, grad_a=ga)
    assert (out == 7).all() and (ga == 7).all() and c.L.stale_call_seen()


def test_lora_repeats_graph_and_streams():
    """Same bytes every time; captured and replayed with new routing; two
    calls at once with workspaces of their own."""
    m = ep()
    c = Case(_ids(400, 1, 6, 3), 6, 512, 520, 16, True, True, seed=3)
    d, ids = c.dev, c.ids.to(DEV)

    def step(L):
        m.ep_layout(ids, 6, out=L)
        out = m.ep_lora(d["x"].nan_to_num(0.0), L, d["a"], d["b"], base=d["base"], **c.kw)
        go = torch.nan_to_num(d["go"], posinf=0.0)
        return (out, *m.ep_lora_backward(go, d["x"].nan_to_num(0.0), L, d["a"], d["b"], **c.kw))

    eager = m.ep_layout(ids, 6, expert_row_src=True)
    first = step(eager)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(step(eager), first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.L)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(c.L)
    for rep in range(4):
        ids.copy_(_ids(400, 1, 6, 30 + rep))
        want = step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))
    lay2 = m.ep_layout(ids, 6, expert_row_src=True)
    want = step(eager)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        one = step(lay2)
    two = step(eager)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one + two, want + want))


def _needs_24_bits(T, E, H, N, R):
    """Inputs whose u and v are 1 + 2^-10 + 2^-20 and -(1 + 2^-10): in every
    result those cancel to a multiple of 2^-20, in some without anything
    larger left.  Each expert has 8 rows of them and zeros else, so that no
    partial sum needs more than 23 bits, in whatever order it is formed."""
    ids = torch.arange(T) % E
    x, go = torch.zeros(T, H), torch.zeros(T, N)
    a, b = torch.zeros(E, R, H), torch.zeros(E, N, R)
    for e in range(E):
        rows = torch.nonzero(ids == e).reshape(-1)
        at = rows[torch.linspace(0, len(rows) - 1, 8).long()]
        for t in (x, go):
            t[at[::2], :3] = torch.tensor([1.0, 2.0**-10, 2.0**-20])
            t[at[1::2], :3] = torch.tensor([-1.0, -(2.0**-10), 0.0])
            t[at, 4] = 1.0
    a[:, 0, :3], a[:, 1, :2], a[:, :2, 8:] = 1.0, -1.0, 1.0
    b[:, :3, 0], b[:, :2, 1], b[:, 8:, :2] = 1.0, -1.0, 1.0
    return ids, *(t.to(torch.bfloat16) for t in (x, go, a, b))


@pytest.mark.parametrize("T,E", [(24, 3), (2600, 3), (4300, 60)])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_lora_inner_products_are_not_rounded(T, E, R):
    """u and v in the second products with all of fp32's 24 bits: every result
    is the bf16 rounding of the exact value."""
    m = ep()
    H, N = 136, 520
    ids, x, go, a, b = _needs_24_bits(T, E, H, N, R)
    L = m.ep_layout(ids[:, None].to(DEV), E, expert_row_src=True)
    dx, dgo, da, db = (t.to(DEV) for t in (x, go, a, b))
    got = [m.ep_lora(dx, L, da, db, gather=True, scatter=True)]
    got += m.ep_lora_backward(dgo, dx, L, da, db, gather=True, scatter=True)
    rows = [np.nonzero(ids.numpy() == e)[0] for e in range(E)]
    rows_of = [(r, r) for r in rows]
    out, _ = LO.lora(f64(x), f64(a), f64(b), np.ones(E), np.zeros((T, N)), rows_of)
    back = LO.lora_backward(f64(go), f64(x), f64(a), f64(b), np.ones(E), np.zeros((T, H)), rows_of)
    live = np.flatnonzero(f64(x)[:, 2])
    assert (out[live][:, 8:] == 2.0**-20).all() and (back[0][0][live][:, 8:] == 2.0**-20).all()
    assert (back[1][0][:, 0, 4] == 2.0**-18).all() and (back[2][0][:, 4, 0] == 2.0**-18).all()
    for name, g, want in zip(("out", "grad_x", "grad_a", "grad_b"), got, [out, *(w for w, _ in back)]):
        want32 = torch.from_numpy(want).to(torch.float32)
        assert torch.equal(want32.double(), torch.from_numpy(want))  # exact in fp32
        assert torch.equal(g.cpu(), want32.to(torch.bfloat16)), name


@pytest.mark.parametrize("R", [8, 32, 64, 128])
def test_lora_inner_products_above_the_largest_bf16(R):
    """u and v between the largest bf16 and the largest fp32 are finite."""
    m = ep()
    H = N = 64
    big, more = float(torch.finfo(torch.bfloat16).max), 1.5 * 2.0**119
    u = big + more
    assert big + 2.0**119 < u < torch.finfo(torch.float32).max
    x = torch.zeros(4, H)
    x[:, 0], x[:, 1] = big, more
    x[1] *= -1
    a, b = torch.zeros(1, R, H), torch.zeros(1, N, R)
    a[0, 0, :2], a[0, 0, 2:] = 1.0, 2.0**-10
    b[0, :2, 0], b[0, 2:, 0] = 1.0, 2.0**-10
    x, a, b = (t.to(torch.bfloat16).to(DEV) for t in (x, a, b))
    L = m.ep_layout(torch.zeros(4, 1, dtype=torch.int64, device=DEV), 1, expert_row_src=True)
    out = m.ep_lora(x, L, a, b, gather=True, scatter=True)
    gx, _, _ = m.ep_lora_backward(x, x, L, a, b, gather=True, scatter=True)
    want = torch.tensor([u, -u, u, u], device=DEV)[:, None].expand(4, N - 2) * 2.0**-10
    assert torch.equal(out[:, 2:], want.to(torch.bfloat16)) and torch.equal(gx[:, 2:], want.to(torch.bfloat16))
    # one row's weight gradients: v x^T and g u^T
    one = m.ep_layout(torch.zeros(1, 1, dtype=torch.int64, device=DEV), 1, expert_row_src=True)
    small = torch.full((1, H), 2.0**-12, dtype=torch.bfloat16, device=DEV)
    _, ga, _ = m.ep_lora_backward(x[:1].clone(), small, one, a, b, gather=True, scatter=True)
    _, _, gb = m.ep_lora_backward(small, x[:1].clone(), one, a, b, gather=True, scatter=True)
    want = (torch.tensor(u, device=DEV) * 2.0**-12).to(torch.bfloat16)
    assert (ga[0, 0] == want).all() and (gb[0, :, 0] == want).all()


def _formula(x, go, a, b, rows):
    """The four results of one expert's rows, in float64 and without a matrix
    product of a library, so that infinities go as the formulas have them."""
    with np.errstate(invalid="ignore"):
        u = (x[rows][:, None, :] * a[None]).sum(2)
        v = (go[rows][:, :, None] * b[None]).sum(1)
        out, gx = (u[:, None, :] * b[None]).sum(2), (v[:, :, None] * a[None]).sum(1)
        ga = (v[:, :, None] * x[rows][:, None, :]).sum(0)
        gb = (go[rows][:, :, None] * u[:, None, :]).sum(0)
    return out, gx, ga, gb


@pytest.mark.parametrize("where", ["a", "b", "x", "go", "a and x", "b and go"])
@pytest.mark.parametrize("R", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("T", [9, 700])
def test_lora_infinite_factors_of_the_second_products(T, R, where):
    """An infinity in B, A, x or grad_out meets u and v whose bf16 parts may be
    zero (small integers): the result is the formula's infinity, NaN only
    where the formula has it (0 times infinity, infinities of both signs), and
    what the infinity does not reach is as without it."""
    m = ep()
    H, N = 72, 136
    g = torch.Generator().manual_seed(R + T)
    ints = lambda *s: torch.randint(1, 4, s, generator=g).float()  # noqa: E731  positive: u and v are not 0
    x, go, a, b = ints(T, H), ints(T, N), ints(1, R, H), ints(1, N, R)
    a[0, R // 2] *= -1  # some u and dx terms negative
    b[0, :, 1] = 0.0  # v of it is 0
    for name in where.split(" and "):
        t = dict(a=a[0], b=b[0], x=x, go=go)[name]
        t[-1, 5], t[0, t.shape[1] - 1] = float("inf"), float("-inf")
    x, go, a, b = (t.to(torch.bfloat16) for t in (x, go, a, b))
    L = m.ep_layout(torch.zeros(T, 1, dtype=torch.int64, device=DEV), 1, expert_row_src=True)
    d = [t.to(DEV) for t in (x, go, a, b)]
    got = [m.ep_lora(d[0], L, d[2], d[3], gather=True, scatter=True)]
    got += m.ep_lora_backward(d[1], d[0], L, d[2], d[3], gather=True, scatter=True)
    want = _formula(f64(x), f64(go), f64(a[0]), f64(b[0]), np.arange(T))
    for name, v, w in zip(("out", "grad_x", "grad_a", "grad_b"), got, want):
        v = f64(v).reshape(w.shape)
        assert np.array_equal(np.isnan(v), np.isnan(w)), name
        inf = np.isinf(w)
        assert np.array_equal(np.isinf(v), inf) and np.array_equal(v[inf], w[inf]), name
        # sums of integers, exact in fp32: below 2^24 but for the gradients of many rows
        fine = np.isfinite(w)
        assert (np.abs(v[fine] - w[fine]) <= (LO.UBF + 2 * T * LO.U32) * np.abs(w[fine]) + T * 2.0**-100).all(), name
    assert any(np.isinf(w).any() for w in want)


@pytest.mark.parametrize("T,K,R", [(135_000, 1, 8), (140_000, 1, 72), (67_000, 2, 24), (136_000, 1, 64)])
def test_lora_backward_more_rows_than_32_chunks_hold(T, K, R):
    """More than 131,072 rows, where the weight gradients' chunks have reached
    4096 rows and their number grows.  Small integers, every sum exact: the
    gradients are the bf16 roundings of the exact values."""
    E, H, N = 4, 24, 16
    ids = _ids(T, K, E, T, none=0.02)
    assert (ids >= 0).sum() > 131_072
    c = Case(ids, E, H, N, R, True, K == 1, seed=R, ints=True)
    gx, ga, gb, want = c.backward()
    for e, (xi, oi) in enumerate(c.rows_of):  # no sum of magnitudes leaves fp32's whole numbers
        u, v = f64(c.x)[xi] @ f64(c.a)[e].T, f64(c.go)[oi] @ f64(c.b)[e]
        assert max((np.abs(v).T @ np.abs(f64(c.x)[xi])).max(), (np.abs(f64(c.go)[oi]).T @ np.abs(u)).max()) < 2**24
    sel = torch.from_numpy(c.selected)
    for name, g, (v, _) in zip("xab", (gx, ga, gb), want):
        v = torch.from_numpy(v).to(torch.float32).to(torch.bfloat16)
        assert torch.equal(g.cpu()[sel] if name == "x" else g.cpu(), v[sel] if name == "x" else v), name
