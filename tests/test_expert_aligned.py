"""Experts' layers over aligned segments: the padding between them takes no
part, neither in what is launched nor in the workspace nor in the limits."""
import ctypes

import pytest
import torch

import test_expert_host as host
import workloads as W
from combine_ep_layout_03_amd import _lib


@pytest.mark.parametrize("T,K,E,H,N", [(4096, 1, 1, 256, 512), (900, 2, 3, 64, 72), (16, 4, 64, 4096, 2048),
                                       (20000, 2, 4, 1024, 1024)])
@pytest.mark.parametrize("A", [2, 128, 1 << 14])
def test_padding_takes_no_workspace(T, K, E, H, N, A):
    lin = host._linear(n_out=N)
    need = lambda a: _lib.lib().ep_expert_linear_workspace_bytes(  # noqa: E731
        ctypes.byref(host._problem(T=T, K=K, E=E, H=H, A=a)), ctypes.byref(lin))
    assert need(A) == need(0) > 0


def test_padding_is_not_counted_against_the_limits():
    """1024 experts aligned to 65,536 rows: 67 million rows of buffer, 128 of a
    selection."""
    p, lin = host._problem(T=16, K=8, E=1024, H=1024, A=1 << 16), host._linear(n_out=1024, act=2)
    assert _lib.lib().ep_expert_linear_workspace_bytes(ctypes.byref(p), ctypes.byref(lin)) == 16
    # past the size checks, and refused for what is wrong with it
    assert host.forward(p=p, lin=lin, x=None) == _lib.EP_EINVAL
    assert host.backward(p=p, lin=lin, go=None) == _lib.EP_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,E,H,N,A", [(16, 4, 64, 1024, 2048, 128), (1, 8, 256, 1032, 264, 16),
                                         (2100, 1, 2, 264, 136, 4096), (4100, 2, 33, 264, 264, 256)])
def test_aligned_equals_unaligned(T, K, E, H, N, A):
    """The same rows in the same order through the same tiles: equal bytes,
    forward and in every gradient."""
    import test_gpu_expert_linear as base

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"aligned T={T} K={K} E={E} H={H} N={N} A={A}", flush=True)
    m, dev = base.ep(), base.DEV
    idx, _ = W.make_routing(W.Workload("a", T=T, H=H, K=K, E=E, mask_p=0.05, seed=T))
    g = torch.Generator().manual_seed(T)
    x, go = base.bf(g, 1.0, T, H).to(dev), base.bf(g, 1.0, T * K, N).to(dev)
    w, b = base.bf(g, H**-0.5, E, 2 * N, H).to(dev), base.bf(g, 0.5, E, 2 * N).to(dev)
    kw = dict(activation=m.EP_ACT_SILU, gated=True, gather=True)
    got = []
    for a in (0, A):
        L = m.ep_layout(idx.to(dev), E, expert_alignment=a, expert_row_src=True)
        rows = L.max_expert_rows()
        at = torch.cat([torch.arange(int(o), int(o) + int(c)) for o, c in zip(L.offsets[:E].cpu(), L.counts[:E].cpu())])
        at = at.to(dev)
        pre = torch.zeros(rows, 2 * N, dtype=torch.bfloat16, device=dev)
        out = m.ep_expert_linear(x, L, w, bias=b, pre=pre, **kw)
        grad = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
        grad[at] = go[: len(at)]
        gx, gw, gb, gp = m.ep_expert_linear_backward(grad, x, L, w, pre=pre, bias=True, **kw)
        got.append((out[at], pre[at], gx[at], gw, gb, gp[at]))
    torch.cuda.synchronize()
    for p, q, name in zip(*got, ("out", "pre", "grad_x", "grad_w", "grad_bias", "grad_pre")):
        assert torch.equal(p, q), name
