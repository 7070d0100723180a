"""GPU parity of the router's balance loss and its gradient against the float64
oracle: counts exact, sums within derived bounds."""
import numpy as np
import pytest
import torch

from oracle import expert_oracle as XO
from oracle.layer_oracle import U32, UBF

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def ep():
    import combine_ep_layout_03_amd as m

    return m


def score_id(score):
    return ep().EP_SCORE_SIGMOID if score == "sigmoid" else ep().EP_SCORE_SOFTMAX


def check(l, idx, score, coef=0.7, seq=None, mask=None, base=True, g=1.5):
    m = ep()
    T, E = l.shape
    K = idx.shape[1]
    print(f"balance T={T} E={E} K={K} {score} {l.dtype} B={1 if seq is None else len(seq) - 1}", flush=True)
    dl, di = l.to(DEV), idx.to(DEV)
    ds = None if seq is None else torch.tensor(seq, dtype=torch.int32, device=DEV)
    dm = None if mask is None else mask.to(DEV)
    kw = dict(score=score_id(score), coef=coef, seq_offsets=ds, token_mask=dm)
    loss, counts, tokens, mean = m.ep_balance_loss(dl, di, **kw)
    l64 = l.double().numpy()
    nm = None if mask is None else mask.numpy().astype(bool)
    wl, wc, wt, wm = XO.balance(l64, idx.numpy(), score, coef, seq, nm)
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(tokens.cpu().numpy(), wt)
    big = XO.share_rtol(np.where(np.isfinite(l64), l64, 0))
    # n additions at most, whatever their order
    tol = wm * (big + (wt[:, None] + 4) * U32) + XO.TINY
    assert (np.abs(mean.cpu().double().numpy() - wm) <= tol).all()
    assert abs(float(loss) - wl) <= abs(wl) * (big + (wt.max(initial=0) + 8) * U32) + XO.TINY
    gb = None
    if base:
        gb = (torch.randn(T, E, generator=torch.Generator().manual_seed(T)) * 1e-3).to(l.dtype)
    gl = torch.tensor([g], device=DEV)
    out = m.ep_balance_loss_backward(gl, dl, counts, tokens, K, grad_base=None if gb is None else gb.to(DEV), **kw)
    assert out.dtype == l.dtype
    want, bound = XO.balance_backward(np.float32(g), l64, wc, wt, K, score, coef, seq, nm,
                                      None if gb is None else gb.double().numpy())
    if l.dtype == torch.bfloat16:
        bound = bound * 1.01 + UBF * np.abs(want)
    err = np.abs(out.cpu().double().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()
    # the same inputs give the same bytes, and the base may be the output
    again = m.ep_balance_loss(dl, di, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, tokens, mean)))
    if gb is not None:
        inplace = gb.to(DEV)
        m.ep_balance_loss_backward(gl, dl, counts, tokens, K, grad_base=inplace, out=inplace, **kw)
        assert torch.equal(inplace, out)
    return loss, counts, tokens, mean


def make(T, E, K, dtype=torch.float32, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed + T * 7 + E)
    l = (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5).to(dtype)
    return l, l.float().topk(K, dim=1).indices


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 64, 4), (64, 63, 3), (200, 65, 8), (37, 256, 8),
                                   (50, 255, 8), (33, 257, 4), (20, 1024, 32), (19, 1023, 2), (1100, 36, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance_shapes(T, E, K, score, dtype):
    check(*make(T, E, K, dtype), score)


@pytest.mark.parametrize("seq", [[0, 100], [0, 0, 100], [3, 16, 16, 17, 80, 99], [0, 32, 48, 64, 64, 64, 100], [50, 50, 50],
                                 [0] + list(range(0, 101))])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_sequences_and_masks(seq, score):
    """Ragged, empty and one-token sequences, tokens of none, masked tokens."""
    l, idx = make(100, 24, 3)
    mask = torch.rand(100, generator=torch.Generator().manual_seed(2)) > 0.2
    check(l, idx, score, seq=seq)
    check(l, torch.where(mask[:, None], idx, -1), score, seq=seq, mask=mask)
    # a masked token's selections do not count
    check(l, idx, score, seq=seq, mask=mask.to(torch.uint8))


def test_balance_many_sequences():
    g = torch.Generator().manual_seed(3)
    l, idx = make(3000, 20, 2)
    cuts = sorted(torch.randint(0, 2991, (700,), generator=g).tolist())
    check(l, idx, "softmax", seq=[0, *cuts, 2990])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_special_logits_and_ids(score):
    l, idx = make(40, 12, 3)
    l[0, 3] = NAN
    l[1] = -INF
    l[2, :11] = -INF
    l[3, 4] = INF
    l[4] = -300.0  # every sigmoid underflows
    l[5] = 300.0
    l[6, 2] = 3e38
    l[7] = NAN
    l[8, 1] = -3e38
    idx[9, 0], idx[9, 1], idx[10] = 12, -7, -1
    idx[11] = 5  # one expert named three times counts three times
    idx[12, 0] = 1 << 40
    check(l, idx, score, base=True)
    out = ep().ep_balance_loss(l.to(DEV), idx.to(DEV), score=score_id(score))
    assert all(torch.isfinite(t.float()).all() for t in out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance_everything_masked_and_no_token(dtype):
    m = ep()
    l, idx = make(30, 16, 2, dtype)
    check(l, idx, "softmax", mask=torch.zeros(30, dtype=torch.bool), seq=[0, 10, 30])
    loss, counts, tokens, mean = m.ep_balance_loss(l[:0].to(DEV), idx[:0].to(DEV))
    assert float(loss) == 0 and (counts == 0).all() and (tokens == 0).all() and (mean == 0).all()
    seq = torch.zeros(4, dtype=torch.int32, device=DEV)
    loss, counts, tokens, mean = m.ep_balance_loss(l[:0].to(DEV), idx[:0].to(DEV), seq_offsets=seq)
    assert counts.shape == (3, 16) and (counts == 0).all() and (tokens == 0).all() and float(loss) == 0
    assert m.ep_balance_loss_backward(loss, l[:0].to(DEV), counts, tokens, 2, seq_offsets=seq).shape == (0, 16)


def test_balance_rows_off_the_vector():
    """Logits, base and result at element alignment only."""
    m = ep()
    l, idx = make(70, 64, 4)
    want = m.ep_balance_loss(l.to(DEV), idx.to(DEV))
    flat = torch.zeros(70 * 64 + 1, device=DEV)
    flat[1:] = l.reshape(-1).to(DEV)
    got = m.ep_balance_loss(flat[1:].view(70, 64), idx.to(DEV))
    assert torch.equal(got[1], want[1])
    # other lanes hold other experts: the same sums in the same order by token
    assert torch.allclose(got[3], want[3], rtol=100 * U32, atol=0)
    g = torch.ones(1, device=DEV)
    a = m.ep_balance_loss_backward(g, l.to(DEV), want[1], want[2], 4)
    b = m.ep_balance_loss_backward(g, flat[1:].view(70, 64), want[1], want[2], 4)
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-6 * float(a.abs().max()))


def test_balance_large_sampled():
    """65,536 x 256 in 16 sequences: counts against torch, the mean and the
    loss against float64 sums on the GPU, gradients of 64 tokens against the
    oracle."""
    m = ep()
    T, E, K = 65536, 256, 8
    g = torch.Generator(device=DEV).manual_seed(9)
    l = torch.randn(T, E, generator=g, device=DEV) * 1.5
    idx = l.topk(K, dim=1).indices.contiguous()
    seq = [0] + sorted(torch.randint(0, T, (15,), generator=torch.Generator().manual_seed(1)).tolist()) + [T - 5]
    ds = torch.tensor(seq, dtype=torch.int32, device=DEV)
    loss, counts, tokens, mean = m.ep_balance_loss(l, idx, score=m.EP_SCORE_SIGMOID, coef=0.01, seq_offsets=ds)
    s = torch.sigmoid(l.double())
    p = s / s.sum(1, keepdim=True)
    total = 0.0
    for b in range(16):
        part = slice(seq[b], seq[b + 1])
        c = torch.bincount(idx[part].reshape(-1), minlength=E)
        n = seq[b + 1] - seq[b]
        assert torch.equal(counts[b].long(), c) and int(tokens[b]) == n
        if n:
            want = p[part].mean(0)
            assert ((mean[b] - want).abs() <= want * (XO.share_rtol(np.array([8.0])) + 300 * U32)).all()
            total += float((c * want).sum()) * E / (K * n) * 0.01 / 16
    assert abs(float(loss) - total) <= total * 1e-5
    gl = torch.tensor([2.0], device=DEV)
    d = m.ep_balance_loss_backward(gl, l, counts, tokens, K, score=m.EP_SCORE_SIGMOID, coef=0.01, seq_offsets=ds)
    b = 15
    at = list(range(seq[b], seq[b + 1], max(1, (seq[b + 1] - seq[b]) // 64)))
    sub = l[at].double().cpu().numpy()
    want = np.zeros_like(sub)
    for i in range(len(at)):
        q, rest = XO.share(sub[i], "sigmoid")
        f = 2.0 * 0.01 * E / (K * 16 * float(tokens[b]) ** 2) * counts[b].cpu().numpy()
        want[i] = q * rest * (f - (f * q).sum())
    err = np.abs(d[at].cpu().double().numpy() - want)
    assert (err <= 1e-5 * np.abs(want).max(1, keepdims=True)).all()
    assert (d[T - 5:] == 0).all()


def test_balance_offsets_past_32_bits():
    """4.3 million tokens x 256 in bf16 (2.2 GB) and a gap: the last tokens as
    in a call of their own."""
    m = ep()
    T, E, K = 4_300_000, 256, 2
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    idx = torch.full((T, K), -1, dtype=torch.int64, device=DEV)
    last, li = make(100, E, K, torch.bfloat16)
    l[-100:], idx[-100:] = last.to(DEV), li.to(DEV)
    seq = torch.tensor([T - 100, T], dtype=torch.int32, device=DEV)
    a = m.ep_balance_loss(l, idx, seq_offsets=seq)
    b = m.ep_balance_loss(last.to(DEV), li.to(DEV))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.allclose(a[3], b[3], rtol=200 * U32, atol=0)
    g = torch.ones(1, device=DEV)
    da = m.ep_balance_loss_backward(g, l, a[1], a[2], K, seq_offsets=seq)
    db = m.ep_balance_loss_backward(g, last.to(DEV), b[1], b[2], K)
    assert torch.equal(da[-100:], db) and not da[:-100].any()


def test_balance_bad_offsets_stay_in_range():
    """Descending offsets and ones past the tokens: no meaning, no fault, and a
    later good call is not touched by it."""
    m = ep()
    l, idx = make(100, 16, 2)
    dl, di = l.to(DEV), idx.to(DEV)
    want = m.ep_balance_loss(dl, di)
    for bad in ([0, 90, 20, 100], [-5, 300], [100, 0], [1 << 30, -(1 << 30), 7]):
        seq = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out = m.ep_balance_loss(dl, di, seq_offsets=seq)
        m.ep_balance_loss_backward(torch.ones(1, device=DEV), dl, out[1], out[2], 2, seq_offsets=seq)
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.ep_balance_loss(dl, di), want))


def test_balance_captured_in_a_graph_twice():
    """Two captured graphs that share a workspace, replayed in turn with eager
    calls between: each replay equals the eager result."""
    m = ep()
    l, idx = make(600, 48, 4)
    dl, di = l.to(DEV), idx.to(DEV)
    seq = torch.tensor([0, 200, 590], dtype=torch.int32, device=DEV)
    ws = torch.empty(m.ep_balance_workspace_bytes(600, 48, 4, 2), dtype=torch.uint8, device=DEV)
    gl = torch.ones(1, device=DEV)

    def step():
        out = m.ep_balance_loss(dl, di, seq_offsets=seq, workspace=ws)
        return (*out, m.ep_balance_loss_backward(gl, dl, out[1], out[2], 4, seq_offsets=seq))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    for k in range(3):
        dl.copy_(make(600, 48, 4, seed=k)[0])
        want = step()
        torch.cuda.synchronize()
        for graph, got in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k
