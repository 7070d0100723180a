"""Refusals of the experts' layers and the balance loss, before any launch: the
header against the library, the C entry points with placeholder pointers that
are never dereferenced, the binding's argument checks, and the workspaces
against splits of the rows and of the tokens (CPU only)."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import combine_ep_layout_03_amd as ep
from combine_ep_layout_03_amd import _lib, expert

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_mi355x_expert.h")
FAR = [ctypes.c_void_p((2 + i) << 40) for i in range(12)]


def at(base, bytes_):
    return ctypes.c_void_p(base.value + bytes_)


def test_header_matches_the_library():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(["ep_expert_linear", "ep_expert_linear_workspace_bytes", "ep_expert_linear_backward",
                            "ep_balance_workspace_bytes", "ep_balance_loss", "ep_balance_loss_backward"])
    for n in names:
        assert hasattr(_lib.lib(), n) and n in _lib.EXPORTS and n in ep.__all__
        assert getattr(expert, n) is getattr(ep, n)
    for n in ("NONE", "RELU", "SILU", "GELU", "GELU_TANH"):
        value = int(re.search(rf"#define EP_ACT_{n} (\d)", open(HEADER).read()).group(1))
        assert getattr(ep, "EP_ACT_" + n) == getattr(_lib, "EP_ACT_" + n) == value


def test_header_compiles_as_c11_and_structs_match(tmp_path):
    from combine_ep_layout_03_amd import build as b

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    sizes = {"ep_linear_t": _lib.Linear, "ep_balance_t": _lib.Balance}
    checks = "".join(f"_Static_assert(sizeof({n}) == {ctypes.sizeof(c)}, \"{n}\");\n" for n, c in sizes.items())
    src = tmp_path / "use.c"
    src.write_text('#include "ep_mi355x_expert.h"\n' + checks +
                   "size_t use(void) { ep_balance_t b = {0}; return ep_balance_workspace_bytes(&b); }\n")
    res = subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-fsyntax-only", *b.C_HIP_FLAGS, "-I",
                          os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def _layout():
    lay = _lib.LayoutStruct()
    for n in ("counts", "offsets", "slot", "status", "expert_row_src"):
        setattr(lay, n, 1 << 20)
    lay.expert_row_capacity = 1 << 30
    return lay


def _problem(T=16, H=256, K=2, E=64, G=0, A=0, flags=0):
    return _lib.Problem(T, H, K, E, G, A, flags)


def _linear(n_out=512, act=0, gated=0, w=FAR[10], bias=None):
    return _lib.Linear(w, bias, n_out, act, gated)


def forward(p=None, lin=None, lay=None, x=FAR[0], ldx=0, res=FAR[1], ldr=0, out=FAR[2], ldo=0, pre=FAR[3], ldp=0):
    p, lin, lay = p or _problem(), lin or _linear(), lay or _layout()
    return _lib.lib().ep_expert_linear(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(lin), x, ldx, res, ldr, out, ldo,
                                       pre, ldp, None)


def backward(p=None, lin=None, lay=None, go=FAR[0], ldgo=0, x=FAR[1], ldx=0, pre=FAR[2], ldp=0, gpre=FAR[3], ldgp=0,
             gx=FAR[4], ldgx=0, gw=FAR[5], gb=FAR[6], ws=FAR[7], nws=1 << 40):
    p, lin, lay = p or _problem(), lin or _linear(act=2), lay or _layout()
    return _lib.lib().ep_expert_linear_backward(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(lin), go, ldgo, x, ldx,
                                                pre, ldp, gpre, ldgp, gx, ldgx, gw, gb, ws, nws, None)


@pytest.mark.parametrize("p,lin,code", [
    (dict(H=260), {}, "ENOTSUP"), ({}, dict(n_out=12), "ENOTSUP"), ({}, dict(n_out=0), "EINVAL"),
    ({}, dict(act=5), "EINVAL"), ({}, dict(act=-1), "EINVAL"), ({}, dict(gated=2), "EINVAL"),
    (dict(flags=1), {}, "EINVAL"), (dict(flags=4), {}, "EINVAL"), (dict(T=1 << 30), {}, "ENOTSUP"),
    (dict(K=33), {}, "ENOTSUP"), (dict(K=0), {}, "EINVAL"), (dict(E=1025), {}, "ENOTSUP"), (dict(T=-1), {}, "EINVAL"),
    (dict(H=(1 << 20) + 8), {}, "ENOTSUP"), ({}, dict(n_out=(1 << 20) + 8), "ENOTSUP"),
    ({}, dict(n_out=(1 << 19) + 8, gated=1), "ENOTSUP"), (dict(H=1 << 16), dict(n_out=1 << 15), "ENOTSUP"),
    (dict(T=1 << 24, H=1 << 11), dict(n_out=1 << 12), "ENOTSUP"),
])
def test_linear_size_refusals(p, lin, code):
    prob, want = _problem(**p), getattr(_lib, "EP_" + code)
    assert forward(p=prob, lin=_linear(**lin)) == want
    assert backward(p=prob, lin=_linear(**{"act": 2, **lin})) == want
    assert _lib.lib().ep_expert_linear_workspace_bytes(ctypes.byref(prob), ctypes.byref(_linear(**lin))) == 0


def test_linear_pointer_stride_and_overlap_refusals():
    off8 = at(FAR[0], 8)
    rows, N, H = 32, 512, 256
    w_bytes = 2 * 64 * 512 * 256
    for kw in (dict(x=None), dict(out=None), dict(x=off8), dict(out=off8), dict(res=off8), dict(pre=off8),
               dict(ldx=248), dict(ldx=260), dict(ldo=504), dict(ldr=516), dict(ldp=508), dict(ldx=(1 << 21) + 8),
               dict(lin=_linear(w=None)), dict(lin=_linear(w=off8)), dict(lin=_linear(bias=off8)),
               dict(out=FAR[0]), dict(out=at(FAR[0], 2 * rows * H - 16)), dict(out=FAR[10]),
               dict(out=at(FAR[10], w_bytes - 16)), dict(pre=FAR[2]), dict(pre=FAR[0]), dict(pre=FAR[1]),
               dict(lin=_linear(bias=FAR[2])), dict(out=FAR[1], ldo=1024), dict(out=at(FAR[1], 2 * N)),
               dict(lay=_lib.LayoutStruct())):
        assert forward(**kw) == _lib.EP_EINVAL, kw
    assert forward(p=_problem(T=0), x=None, out=None, res=None, pre=None) == _lib.EP_OK
    bare = _layout()
    bare.expert_row_src = None
    short = _layout()
    short.expert_row_capacity = 31
    for lay in (bare, short):
        assert forward(p=_problem(flags=_lib.EP_FLAG_GATHER_ROWS), lay=lay) == _lib.EP_EINVAL
    # a gathered token matrix beyond 64 GiB
    big = _problem(T=(1 << 16) + 1, H=8, K=1, E=1, flags=_lib.EP_FLAG_GATHER_ROWS)
    assert forward(p=big, lin=_linear(n_out=8), ldx=1 << 19) == _lib.EP_ENOTSUP


def test_linear_backward_refusals():
    p = _problem()
    need = _lib.lib().ep_expert_linear_workspace_bytes(ctypes.byref(p), ctypes.byref(_linear()))
    assert need == 16
    off8 = at(FAR[0], 8)
    for kw in (dict(go=None), dict(x=None), dict(pre=None), dict(gpre=None), dict(go=off8), dict(gx=off8), dict(gw=off8),
               dict(gb=off8), dict(gw=None), dict(ldgo=504), dict(ldgx=248), dict(ldp=508), dict(ws=None), dict(ws=off8),
               dict(lin=_linear(act=2, w=None)), dict(gpre=FAR[0]), dict(gpre=FAR[1]), dict(gpre=FAR[10]),
               dict(gpre=at(FAR[2], 1024)), dict(gpre=FAR[2], ldgp=1024), dict(gx=FAR[0]), dict(gx=FAR[1]),
               dict(gx=FAR[2]), dict(gx=FAR[3]), dict(gx=FAR[10]), dict(gx=FAR[5]), dict(gw=FAR[0]), dict(gw=FAR[1]),
               dict(gw=FAR[2]), dict(gw=FAR[3]), dict(gw=FAR[10]), dict(gb=FAR[5]), dict(gb=FAR[0]), dict(gb=FAR[3]),
               dict(lin=_linear(act=0)),  # nothing to go through, but pre given
               dict(lin=_linear(act=0), pre=None), dict(lay=_lib.LayoutStruct())):
        assert backward(**kw) == _lib.EP_EINVAL, kw
    # few experts, many rows: a workspace that must be there and apart
    p, lin = _problem(T=4096, K=1, E=1), _linear(act=2)
    need = _lib.lib().ep_expert_linear_workspace_bytes(ctypes.byref(p), ctypes.byref(lin))
    assert need > 16
    assert backward(p=p, lin=lin, nws=need - 1) == _lib.EP_EWORKSPACE
    for ws in (*FAR[:7], FAR[10], at(FAR[5], -need + 16)):
        assert backward(p=p, lin=lin, ws=ws, nws=need) == _lib.EP_EINVAL, ws


def test_linear_workspace_to_the_byte():
    """As the kernels index it: S parts of fp32 [E, W, H] and, behind them, of
    [E, W]; S at its least cost in us, with 64 rows an even share left each and
    no more blocks than fill the chip twice."""
    rng = random.Random(2)
    for _ in range(400):
        T, K, E = rng.randint(1, 20000), rng.randint(1, 4), rng.randint(1, 40)
        H, N, gated = 8 * rng.randint(1, 300), 8 * rng.randint(1, 300), rng.randint(0, 1)
        W = N * (1 + gated)
        tiles = -(-W // 256) * -(-H // 256) * E
        p, lin = _problem(T=T, H=H, K=min(K, E), E=E), _linear(n_out=N, gated=gated)
        rows = T * min(K, E)

        def cost(s):
            steps = -(-(-(-rows // (E * s))) // 32)
            c = float(-(-tiles * s // 256)) * (0.9 * float(steps) + 8.0)
            return c + (5.0 + 8.0 * float((W * H + W) * E * s) / 6.0e6) if s > 1 else c

        tried, s = [], 1
        while s == 1 or (s * tiles <= 512 and 64 * s <= rows // E):
            tried.append(s)
            s += 1 if s < 8 else s // 8
        S = min(tried, key=cost)
        want = S * E * W * (H + 1) * 4 if S > 1 else 16
        got = _lib.lib().ep_expert_linear_workspace_bytes(ctypes.byref(p), ctypes.byref(lin))
        assert got == want
        # the parts of an expert's rows cover them, each once
        cnt = rng.randint(0, T)
        per = -(-(-(-cnt // S)) // 32) * 32
        assert sum(min(per, cnt - min(cnt, per * s)) for s in range(S)) == cnt


def _balance(**kw):
    d = dict(T=16, E=64, K=4, score=0, logits=0, B=3, coef=1.0)
    d.update(kw)
    return _lib.Balance(*d.values())


def loss(b=None, l=FAR[0], i=FAR[1], seq=FAR[2], mask=FAR[3], out=FAR[4], c=FAR[5], t=FAR[6], m=FAR[7], ws=FAR[8],
         nws=1 << 40):
    b = b or _balance()
    return _lib.lib().ep_balance_loss(ctypes.byref(b), l, i, seq, mask, out, c, t, m, ws, nws, None)


def loss_backward(b=None, g=FAR[0], l=FAR[1], seq=FAR[2], mask=FAR[3], c=FAR[4], t=FAR[5], base=FAR[6], out=FAR[7]):
    b = b or _balance()
    return _lib.lib().ep_balance_loss_backward(ctypes.byref(b), g, l, seq, mask, c, t, base, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(E=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(K=65), "EINVAL"), (dict(K=33), "ENOTSUP"),
    (dict(E=1025), "ENOTSUP"), (dict(score=2), "EINVAL"), (dict(logits=2), "EINVAL"), (dict(B=0), "EINVAL"),
    (dict(B=65537), "ENOTSUP"), (dict(coef=float("nan")), "EINVAL"), (dict(coef=float("inf")), "EINVAL"),
    (dict(T=1 << 29), "ENOTSUP"),
])
def test_balance_size_refusals(kw, code):
    b, want = _balance(**kw), getattr(_lib, "EP_" + code)
    assert loss(b) == want and loss_backward(b) == want
    assert _lib.lib().ep_balance_workspace_bytes(ctypes.byref(b)) == 0


def test_balance_pointer_and_overlap_refusals():
    odd = at(FAR[0], 2)
    need = _lib.lib().ep_balance_workspace_bytes(ctypes.byref(_balance()))
    for kw in (dict(l=None), dict(i=None), dict(seq=None), dict(out=None), dict(c=None), dict(t=None), dict(m=None),
               dict(ws=None), dict(l=odd), dict(i=at(FAR[1], 4)), dict(seq=odd), dict(out=odd), dict(c=odd), dict(m=odd),
               dict(ws=at(FAR[8], 8)), dict(out=FAR[0]), dict(c=FAR[1]), dict(t=FAR[2]), dict(m=FAR[3]), dict(m=FAR[5]),
               dict(c=at(FAR[0], 16 * 64 * 4 - 4)), dict(ws=FAR[0]), dict(ws=at(FAR[5], -need + 16)),
               dict(out=at(FAR[6], 8))):
        assert loss(**kw) == _lib.EP_EINVAL, kw
    assert loss(nws=need - 1) == _lib.EP_EWORKSPACE
    for kw in (dict(g=None), dict(l=None), dict(seq=None), dict(c=None), dict(t=None), dict(out=None), dict(g=odd),
               dict(l=odd), dict(base=odd), dict(out=odd), dict(out=FAR[1]), dict(out=FAR[4]), dict(out=FAR[0]),
               dict(out=FAR[2]), dict(out=FAR[3]), dict(out=FAR[5]), dict(out=at(FAR[6], 256))):
        assert loss_backward(**kw) == _lib.EP_EINVAL, kw
    assert loss_backward(_balance(T=0), g=None, l=None, c=None, t=None, out=None) == _lib.EP_OK


def test_balance_workspace_holds_every_part():
    """Slots of (chunk, sequence) parts as the kernels number them: c + b is
    used once and stays below chunks + B, whatever the sequences."""
    rng = random.Random(3)
    for _ in range(200):
        T, E, B = rng.choice([rng.randint(1, 400), rng.randint(400, 100_000)]), rng.randint(1, 300), rng.randint(1, 400)
        chunk = 16
        while T // chunk > 1024:
            chunk *= 2
        slots = -(-T // chunk) + B
        up = lambda n: -(-n // 16) * 16  # noqa: E731
        b = _balance(T=T, E=E, K=1, B=B)
        assert _lib.lib().ep_balance_workspace_bytes(ctypes.byref(b)) == 2 * up(slots * E * 4) + up(slots * 4) + 16
        off = sorted(rng.randint(0, T) for _ in range(B + 1))
        used = set()
        for s in range(B):
            if off[s + 1] > off[s]:
                for c in range(off[s] // chunk, (off[s + 1] - 1) // chunk + 1):
                    assert c + s not in used and c + s < slots
                    used.add(c + s)


def test_binding_refusals():
    z = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    lay = ep.Layout(4, 2, 3, 0, *(z(4, dtype=torch.int32) for _ in range(4)))
    with pytest.raises(ValueError, match=r"w must be"):
        ep.ep_expert_linear(z(8, 16, **bf), lay, z(8, 16, **bf))
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_expert_linear(z(8, 16, **bf), lay, z(3, 8, 16, **bf))
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_expert_linear_backward(z(8, 8, **bf), z(8, 16, **bf), lay, z(3, 8, 16, **bf))
    with pytest.raises(ValueError, match=r"topk_idx must be"):
        ep.ep_balance_loss(z(4, 8), z(8, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_balance_loss(z(4, 8), z(4, 2, dtype=torch.int64))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ep.ep_balance_loss_backward(z(1), z(4, 8, dtype=torch.float64), z(1, 8), z(1), 2)
    stale = lay.handle()
    lay.generation += 1
    with pytest.raises(ep.StaleLayoutError if hasattr(ep, "StaleLayoutError") else RuntimeError):
        ep.ep_expert_linear(z(8, 16, **bf), stale, z(3, 8, 16, **bf))
    assert ep.ep_expert_linear_workspace_bytes(lay, 16, 16) == 16
    assert ep.ep_expert_linear_workspace_bytes(lay, 12, 16) == 0
    assert ep.ep_balance_workspace_bytes(100, 64, 4) > 0 and ep.ep_balance_workspace_bytes(100, 64, 65) == 0
    for sizes in (((1 << 32) + 16, 16), (16, (1 << 32) + 16)):
        with pytest.raises(ValueError, match="int32"):
            ep.ep_expert_linear_workspace_bytes(lay, *sizes)
    with pytest.raises(ValueError, match="int32"):
        ep.ep_balance_workspace_bytes(100, (1 << 32) + 8, 4)
