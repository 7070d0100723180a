"""The experts' layers at sizes that take each tile height, forward and in
both gradients, against the float64 oracle; which height a size takes is read
from the launch plans themselves, on the CPU."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import test_gpu_expert_linear as base
import workloads as W
from oracle import expert_oracle as XO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = base.DEV

# (sub-tiles of 32 rows of a wave, by product: forward, grad_x, grad_w) of each
# size; 0: the kernel for few rows.  About 250 rows an expert and contractions
# of 8 steps and more, with tails: every ring wraps.
LAYERS = [
    ((2, 2, 2), dict(T=2400, K=2, E=33, H=264, N=328, kind="silu", gated=True)),
    ((2, 4, 4), dict(T=4800, K=2, E=33, H=520, N=264, kind="relu", gather=True)),
    ((4, 2, 2), dict(T=4100, K=2, E=33, H=264, N=264, kind="silu", gated=True, gather=True, extra=8)),
    ((4, 4, 4), dict(T=13000, K=1, E=3, H=776, N=520, kind="gelu_tanh")),
    ((4, 5, 4), dict(T=8200, K=2, E=64, H=520, N=264, kind="gelu", gather=True)),
    ((4, 5, 4), dict(T=6000, K=2, E=48, H=776, N=328, kind="none")),
    ((5, 2, 2), dict(T=7000, K=2, E=56, H=520, N=392, kind="gelu_tanh", gated=True, extra=64)),
    ((5, 4, 4), dict(T=8200, K=2, E=64, H=264, N=264, kind="gelu", gated=True)),
    ((5, 4, 4), dict(T=8200, K=2, E=64, H=264, N=520, kind="silu", gather=True)),
]
# gated or not, at each height
FORWARD = [
    (2, dict(T=2400, K=2, E=33, N=328, gated=True)), (4, dict(T=4100, K=2, E=33, N=264, gated=True)),
    (5, dict(T=8200, K=2, E=64, N=264, gated=True)), (2, dict(T=4800, K=2, E=33, N=264, gated=False)),
    (4, dict(T=8200, K=2, E=64, N=264, gated=False)), (5, dict(T=8200, K=2, E=64, N=520, gated=False)),
]
gpu = pytest.mark.gpu


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def _plans(tmp_path, sizes):
    """(forward, grad_x, grad_w, whether together) of each (rows, E, H, N,
    gated), by a program over the launch plans."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "p.cpp").write_text("""
#include <stdio.h>
#include "ep_linear_plan.h"
int main() {
  long rows;
  int E, H, N, gated;
  while (scanf("%ld %d %d %d %d", &rows, &E, &H, &N, &gated) == 5) {
    const int W = gated ? 2 * N : N;
    const auto g = ep::plan_grads(rows, E, H, W, ep::linear_geom(rows, E, H, W).splits, true, true);
    printf("%d %d %d %d\\n", ep::plan_forward(rows, E, N, gated).mi, g.x.mi, g.w.mi, g.together);
  }
}
""")
    exe = tmp_path / "p"
    res = subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I",
                          os.path.join(ROOT, "combine_ep_layout_03_amd", "csrc"), str(tmp_path / "p.cpp"), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    text = "".join("%d %d %d %d %d\n" % s for s in sizes)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    return [tuple(int(v) for v in line.split()) for line in out.splitlines()]


def test_sizes_take_the_heights_they_are_meant_for(tmp_path):
    sizes = [(s["T"] * s["K"], s["E"], s["H"], s["N"], s.get("gated", False)) for _, s in LAYERS]
    assert _plans(tmp_path, sizes) == [(*want, 1) for want, _ in LAYERS]
    sizes = [(s["T"] * s["K"], s["E"], 72, s["N"], s["gated"]) for _, s in FORWARD]
    assert [p[0] for p in _plans(tmp_path, sizes)] == [want for want, _ in FORWARD]


@gpu
@pytest.mark.parametrize("heights,size", LAYERS, ids=lambda v: "-".join(map(str, v)) if isinstance(v, tuple) else "")
def test_every_height_against_the_oracle(heights, size, device):
    """Forward with bias, residual and pre, and the gradients in one launch."""
    base.check(**size)


@gpu
@pytest.mark.parametrize("heights,size", LAYERS, ids=lambda v: "-".join(map(str, v)) if isinstance(v, tuple) else "")
def test_every_height_together_equals_alone(heights, size, device):
    wide = size["N"] * (2 if size.get("gated") else 1)  # the products are those of a bare layer this wide
    base.test_linear_gradients_together_equal_each_alone(size["T"], size["K"], size["E"], size["H"], wide,
                                                         size.get("gather", False))


@gpu
@pytest.mark.parametrize("height,size", FORWARD)
@pytest.mark.parametrize("kind", XO.ACTS)
def test_every_activation_at_every_height(height, size, kind, device):
    """With bias, residual, pre and gathered rows or not in turn; every row
    within the bound of the first and last rows of each tile and a sample."""
    T, K, E, N, gated = (size[k] for k in ("T", "K", "E", "N", "gated"))
    H, gather = 72, kind in ("silu", "none")
    print(f"tiles {height} {size} {kind}", flush=True)
    m = base.ep()
    idx, _ = W.make_routing(W.Workload("x", T=T, H=H, K=K, E=E, mask_p=0.05, seed=T))
    L = m.ep_layout(idx.to(DEV), E, expert_row_src=True)
    rows, wide = L.max_expert_rows(), (2 * N if gated else N)
    g = torch.Generator().manual_seed(len(kind) + N)
    x, res = base.bf(g, 1.0, T if gather else rows, H).to(DEV), base.bf(g, 1.0, rows, N).to(DEV)
    w, b = base.bf(g, 1.5 * H**-0.5, E, wide, H).to(DEV), base.bf(g, 0.5, E, wide).to(DEV)
    out, pre = base.marked(rows, N), base.marked(rows, wide)
    m.ep_expert_linear(x, L, w, bias=b, activation=base.act_id(kind), gated=gated, residual=res, gather=gather, out=out,
                       pre=pre)
    torch.cuda.synchronize()
    rng = np.random.default_rng(7)
    who = []
    for xi, oi in base.rows_of(L, gather):
        n = len(oi)
        at = np.unique(np.concatenate([np.arange(min(n, 3)), np.arange(max(0, n - 3), n), rng.integers(0, max(n, 1), 20)]))
        at = at[at < n]
        who.append((xi[at], oi[at]))
    want, bound, zwant, zbound = XO.linear(base.f64(x), base.f64(w), base.f64(b), kind, gated, base.f64(res), who)
    at = np.concatenate([o for _, o in who])
    assert len(at) > 20 * E / 2
    assert (np.abs(base.f64(out)[at] - want[at]) <= bound[at]).all()
    assert (np.abs(base.f64(pre)[at] - zwant[at]) <= zbound[at]).all()
    # every row of a selection is written, none beside
    live = np.zeros(rows, bool)
    live[: L.num_rows()] = True
    assert not np.isnan(base.f64(out)[live]).any() and not np.isnan(base.f64(pre)[live]).any()
    assert (base.u16(out)[~live] == 0xFFFF).all() and (base.u16(pre)[~live] == 0xFFFF).all()


@gpu
def test_last_rows_past_32_bits_within_the_bound(device):
    """Rows whose byte offsets pass 2^32, in tiles of 320 rows: the last ones
    against float64, as sums in any order."""
    m = base.ep()
    T, H, N, E = 150_000, 16_384, 64, 3
    idx = torch.zeros(T, 1, dtype=torch.int64, device=DEV)
    idx[-50:] = 2
    L = m.ep_layout(idx, E, expert_row_src=True)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(14)
    x[-50:] = torch.randn(50, H, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(E, N, H, generator=g, device=DEV) * H**-0.5).to(torch.bfloat16)
    who = [(np.zeros(0, int),) * 2, (np.zeros(0, int),) * 2, (np.arange(50),) * 2]
    want, bound, _, _ = XO.linear(base.f64(x[-50:]), base.f64(w), None, "none", False, np.zeros((50, N)), who)
    for gather in (False, True):
        y = m.ep_expert_linear(x, L, w, gather=gather)
        assert (np.abs(base.f64(y[-50:]) - want) <= bound).all()
        assert not y[:-50].any()


@gpu
def test_grad_x_alone_takes_no_workspace(device):
    """Rows enough that the weight gradient would be split: grad_x alone
    allocates itself and no parts, and is the same."""
    m = base.ep()
    T, H, N = 16384, 1024, 1024
    L = m.ep_layout(torch.zeros(T, 1, dtype=torch.int64, device=DEV), 1)
    parts = m.ep_expert_linear_workspace_bytes(L, H, N)
    assert parts > 16 << 20
    g = torch.Generator().manual_seed(3)
    x, go, w = base.bf(g, 1.0, T, H).to(DEV), base.bf(g, 1.0, T, N).to(DEV), base.bf(g, 0.1, 1, N, H).to(DEV)
    want = m.ep_expert_linear_backward(go, x, L, w)[0]
    got = torch.zeros_like(want)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    m.ep_expert_linear_backward(go, x, L, w, grad_x=got, needs=(True, False))
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    assert torch.equal(got, want)
    # one that is too small for the parts is no matter either
    got.zero_()
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    m.ep_expert_linear_backward(go, x, L, w, grad_x=got, needs=(True, False), workspace=small)
    assert torch.equal(got, want)
    with pytest.raises(m.EPError):
        m.ep_expert_linear_backward(go, x, L, w, needs=(False, True), workspace=small)
