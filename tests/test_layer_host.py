"""Refusals of the layer operators (router, gradients, adapters), before any
launch: the header against the library, the C entry points with placeholder
pointers that are never dereferenced, and the binding's argument checks (CPU
only)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import combine_ep_layout_03_amd as ep
from combine_ep_layout_03_amd import _lib, layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_mi355x_layer.h")
PTR = ctypes.c_void_p(1 << 20)
FAR = [ctypes.c_void_p((2 + i) << 40) for i in range(8)]


def _declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", src)))


def test_header_matches_the_library():
    names = _declared()
    assert names == sorted(["ep_route", "ep_route_backward", "ep_combine_backward", "ep_lora_workspace_bytes",
                            "ep_lora", "ep_lora_backward"])
    for n in names:
        assert hasattr(_lib.lib(), n) and n in _lib.EXPORTS and n in ep.__all__


def test_header_compiles_as_c99_and_structs_match(tmp_path):
    from combine_ep_layout_03_amd import build as b

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    sizes = {"ep_router_t": _lib.Router, "ep_lora_weights_t": _lib.LoraWeights, "ep_problem_t": _lib.Problem}
    checks = "".join(f"_Static_assert(sizeof({n}) == {ctypes.sizeof(c)}, \"{n}\");\n" for n, c in sizes.items())
    src = tmp_path / "use.c"
    src.write_text('#include "ep_mi355x_layer.h"\n' + checks +
                   "int use(void) { ep_router_t r = {0}; return ep_route(&r, 0, 0, 0, 0, 0, 0); }\n")
    res = subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-fsyntax-only", *b.C_HIP_FLAGS, "-I",
                          os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def _route(**kw):
    r = dict(T=16, E=64, K=4, score=0, logits=0, G=0, TG=0, gtop=1, renorm=0, scale=1.0)
    r.update(kw)
    return _lib.Router(*r.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(E=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(K=65), "EINVAL"),
    (dict(K=33), "ENOTSUP"), (dict(E=1025, K=4), "ENOTSUP"), (dict(score=2), "EINVAL"), (dict(logits=2), "EINVAL"),
    (dict(renorm=2), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(G=7, TG=1), "EINVAL"), (dict(G=-1, TG=1), "EINVAL"), (dict(G=8, TG=0), "EINVAL"),
    (dict(G=8, TG=9), "EINVAL"), (dict(G=8, TG=1, gtop=3), "EINVAL"), (dict(G=32, TG=1, K=4), "EINVAL"),
    (dict(E=130, G=65, TG=65), "ENOTSUP"), (dict(T=1 << 29), "ENOTSUP"),
])
def test_route_refusals(kw, code):
    r = _route(**kw)
    f = FAR
    assert _lib.lib().ep_route(ctypes.byref(r), f[0], None, None, f[1], f[2], None) == getattr(_lib, "EP_" + code)
    if not any(k in kw for k in ("G", "TG", "gtop")):
        assert _lib.lib().ep_route_backward(ctypes.byref(r), f[0], f[1], f[2], f[3], None) == getattr(_lib, "EP_" + code)


def test_route_pointer_refusals():
    L, f, r = _lib.lib(), FAR, _route()
    odd = ctypes.c_void_p((1 << 41) + 2)
    for args in ([None, None, None, f[1], f[2]], [f[0], None, None, None, f[2]], [f[0], None, None, f[1], None],
                 [odd, None, None, f[1], f[2]], [f[0], odd, None, f[1], f[2]],
                 [f[0], None, None, ctypes.c_void_p((1 << 41) + 4), f[2]], [f[0], None, None, f[1], odd]):
        assert L.ep_route(ctypes.byref(r), *args, None) == _lib.EP_EINVAL
    assert L.ep_route(None, f[0], None, None, f[1], f[2], None) == _lib.EP_EINVAL
    # the gradient must not be written over the logits
    assert L.ep_route_backward(ctypes.byref(r), f[0], f[1], f[2], f[0], None) == _lib.EP_EINVAL
    # no tokens: nothing to do, nothing launched
    z = _route(T=0)
    assert L.ep_route(ctypes.byref(z), None, None, None, None, None, None) == _lib.EP_OK
    assert L.ep_route_backward(ctypes.byref(z), None, None, None, None, None) == _lib.EP_OK


def _layout():
    lay = _lib.LayoutStruct()
    for n in ("counts", "offsets", "slot", "status", "expert_row_src"):
        setattr(lay, n, 1 << 20)
    lay.expert_row_capacity = 1 << 30
    return lay


def test_combine_backward_refusals():
    L, f, lay = _lib.lib(), FAR, _layout()
    p = _lib.Problem(16, 256, 4, 64, 0, 0, 0)
    ok = [f[0], f[1], f[2], 64, f[3], f[4]]

    def call(i=None, v=None, prob=p, lay=lay):
        a = list(ok)
        if i is not None:
            a[i] = v
        return L.ep_combine_backward(ctypes.byref(prob), ctypes.byref(lay), *a, None)

    odd = ctypes.c_void_p((1 << 42) + 1)
    for i, v in ((0, None), (1, None), (2, None), (3, -1), (4, None), (5, None), (0, odd), (1, odd), (4, odd),
                 (4, f[2]), (4, f[1])):
        assert call(i, v) == _lib.EP_EINVAL, (i, v)
    assert call(prob=_lib.Problem(16, 256, 33, 64, 0, 0, 0)) == _lib.EP_ENOTSUP
    assert call(prob=_lib.Problem(16, 256, 0, 64, 0, 0, 0)) == _lib.EP_EINVAL
    assert call(lay=_lib.LayoutStruct()) == _lib.EP_EINVAL
    assert call(prob=_lib.Problem(0, 256, 4, 64, 0, 0, 0)) == _lib.EP_OK


def _weights(rank=16, n_out=512, flags=0, a=FAR[5], b=FAR[6], scales=None):
    return _lib.LoraWeights(a, b, scales, rank, n_out, flags)


@pytest.mark.parametrize("p,w,code", [
    (dict(H=260), {}, "ENOTSUP"), ({}, dict(n_out=12), "ENOTSUP"), ({}, dict(rank=12), "ENOTSUP"),
    ({}, dict(rank=136), "ENOTSUP"), ({}, dict(rank=0), "EINVAL"), ({}, dict(n_out=0), "EINVAL"),
    ({}, dict(flags=2), "EINVAL"), (dict(K=4), dict(flags=1), "EINVAL"), (dict(flags=8), {}, "EINVAL"),
    (dict(T=1 << 29), {}, "ENOTSUP"), ({}, dict(a=None), "EINVAL"), ({}, dict(b=None), "EINVAL"),
    ({}, dict(a=ctypes.c_void_p((1 << 42) + 8)), "EINVAL"), ({}, dict(scales=ctypes.c_void_p((1 << 42) + 2)), "EINVAL"),
])
def test_lora_refusals(p, w, code):
    d = dict(T=16, H=256, K=1, E=64, G=0, A=0, flags=0)
    d.update(p)
    prob, wt, lay, f, L = _lib.Problem(*d.values()), _weights(**w), _layout(), FAR, _lib.lib()
    want = getattr(_lib, "EP_" + code)
    big = 1 << 40
    got = L.ep_lora(ctypes.byref(prob), ctypes.byref(lay), ctypes.byref(wt), f[0], 0, f[1], 0, f[2], 0, f[3], big, None)
    assert got == want
    got = L.ep_lora_backward(ctypes.byref(prob), ctypes.byref(lay), ctypes.byref(wt), f[0], 0, f[1], 0, None, 0, f[2], 0,
                             f[3], f[4], f[7], big, None)
    assert got == want
    if not ({"a", "b", "scales"} & set(w)):
        assert L.ep_lora_workspace_bytes(ctypes.byref(prob), ctypes.byref(wt), 0) == 0


def test_lora_strides_overlaps_and_workspace():
    L, f, lay = _lib.lib(), FAR, _layout()
    p, w = _lib.Problem(16, 256, 1, 64, 0, 0, 0), _weights()
    need = L.ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), 0)
    assert need > 0 and L.ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), 1) > need

    def call(x=f[0], ldx=0, base=f[1], ldb=0, out=f[2], ldo=0, ws=f[3], nws=need, lay=lay, p=p):
        return L.ep_lora(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(w), x, ldx, base, ldb, out, ldo, ws, nws, None)

    off8 = ctypes.c_void_p(FAR[0].value + 8)
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(x=off8), dict(out=off8), dict(base=off8),
               dict(ldx=248), dict(ldx=260), dict(ldo=504), dict(ldb=516), dict(ws=off8),
               dict(out=f[0]),  # over x
               dict(out=f[5]), dict(out=f[6]),  # over the adapters
               dict(out=f[1], ldo=1024),  # base's memory with another stride
               dict(out=ctypes.c_void_p(FAR[1].value + 1024))):  # base, one row further
        assert call(**kw) == _lib.EP_EINVAL, kw
    assert call(nws=need - 1) == _lib.EP_EWORKSPACE
    assert call(lay=_lib.LayoutStruct()) == _lib.EP_EINVAL
    # gathered or scattered rows need the layout's row map, long enough
    bare = _layout()
    bare.expert_row_src = None
    assert call(lay=bare, p=_lib.Problem(16, 256, 1, 64, 0, 0, _lib.EP_FLAG_GATHER_ROWS)) == _lib.EP_EINVAL
    short = _layout()
    short.expert_row_capacity = 15
    assert call(lay=short, p=_lib.Problem(16, 256, 1, 64, 0, 0, _lib.EP_FLAG_GATHER_ROWS)) == _lib.EP_EINVAL


def test_lora_backward_overlaps_and_workspace():
    L, f, lay = _lib.lib(), FAR, _layout()
    p, w = _lib.Problem(16, 256, 1, 64, 0, 0, 0), _weights()
    need = L.ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), 1)
    base = ctypes.c_void_p(11 << 40)

    def call(go=f[0], x=f[1], gbase=base, gx=f[2], ga=f[3], gb=f[4], ws=f[7], nws=need):
        return L.ep_lora_backward(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(w), go, 0, x, 0, gbase, 0, gx, 0, ga, gb,
                                  ws, nws, None)

    for kw in (dict(go=None), dict(x=None), dict(gx=None), dict(ga=None), dict(gb=None), dict(ws=None),
               dict(gx=f[1]), dict(gx=f[0]), dict(ga=f[5]), dict(gb=f[6]), dict(ga=f[2]), dict(gb=f[3]),
               dict(gbase=f[3]), dict(gbase=ctypes.c_void_p(FAR[2].value + 512))):
        assert call(**kw) == _lib.EP_EINVAL, kw
    assert call(nws=need - 1) == _lib.EP_EWORKSPACE


def test_outputs_over_inputs_and_each_other():
    L, f, r = _lib.lib(), FAR, _route()  # 16 x 64 logits of 4 bytes, 16 x 4 selections

    def at(base, bytes_):
        return ctypes.c_void_p(base.value + bytes_)

    last = at(f[0], 16 * 64 * 4 - 8)
    for args in ([f[0], None, None, f[0], f[2]], [f[0], None, None, last, f[2]], [f[0], None, None, f[1], last],
                 [f[0], f[1], None, f[1], f[2]], [f[0], None, at(f[2], 255), f[1], f[2]],
                 [f[0], None, None, f[1], at(f[1], 508)]):
        assert L.ep_route(ctypes.byref(r), *args, None) == _lib.EP_EINVAL, args
    for args in ([f[0], f[1], f[2], f[1]], [f[0], f[1], f[2], at(f[2], 252)]):
        assert L.ep_route_backward(ctypes.byref(r), *args, None) == _lib.EP_EINVAL, args
    lay, p = _layout(), _lib.Problem(16, 256, 4, 64, 0, 0, 0)
    for w, go, y, gy, gw in ([f[0], f[1], f[2], f[3], f[0]], [f[0], f[1], f[2], f[3], f[1]], [f[0], f[1], f[2], f[3], f[2]],
                             [f[0], f[1], f[2], f[3], f[3]], [f[0], f[1], f[2], f[0], f[4]]):
        assert L.ep_combine_backward(ctypes.byref(p), ctypes.byref(lay), w, go, y, 64, gy, gw, None) == _lib.EP_EINVAL
    p, w = _lib.Problem(16, 256, 1, 64, 0, 0, 0), _weights()
    need = [L.ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), b) for b in (0, 1)]
    for ws in (f[0], f[1], f[2], f[5], f[6], at(f[0], -need[0] + 16)):
        assert L.ep_lora(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(w), f[0], 0, f[1], 0, f[2], 0, ws, need[0],
                         None) == _lib.EP_EINVAL, ws
    gbase = ctypes.c_void_p(11 << 40)
    for ws in (f[0], f[1], f[2], f[3], f[4], f[5], f[6], gbase, at(f[3], -need[1] + 16)):
        assert L.ep_lora_backward(ctypes.byref(p), ctypes.byref(lay), ctypes.byref(w), f[0], 0, f[1], 0, gbase, 0, f[2], 0,
                                  f[3], f[4], ws, need[1], None) == _lib.EP_EINVAL, ws


def test_binding_keeps_int32_fields_whole():
    for fields in ((4, 8, 2, 0, 0, 1 << 32, 0, 1, 0, 1.0), (4, 8, 2, 1 << 32, 0, 0, 0, 1, 0, 1.0),
                   (4, (1 << 32) + 8, 2, 0, 0, 0, 0, 1, 0, 1.0)):
        with pytest.raises(ValueError, match="int32"):
            layer._router_struct(*fields)
    lay = ep.Layout(4, 2, 3, 0, *(torch.zeros(4, dtype=torch.int32) for _ in range(4)))
    for sizes in (((1 << 32) + 16, 16, 8), (16, (1 << 32) + 16, 8), (16, 16, (1 << 32) + 8)):
        with pytest.raises(ValueError, match="int32"):
            ep.ep_lora_workspace_bytes(lay, *sizes)


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route(z(4, 8), 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ep.ep_route(z(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match=r"\[T, E\]"):
        ep.ep_route(z(8), 2)
    with pytest.raises(ValueError, match=r"topk_idx must be"):
        ep.ep_route_backward(z(4, 2), z(4, 8), z(8, dtype=torch.int64))
    lay = ep.Layout(4, 2, 3, 0, *(z(4, dtype=torch.int32) for _ in range(4)))
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_combine_backward(z(4, 8, dtype=torch.bfloat16), z(8, 8, dtype=torch.bfloat16), lay, z(4, 2))
    with pytest.raises(ValueError, match=r"a must be \[E, R, H\]"):
        ep.ep_lora(z(8, 16), lay, z(8, 16), z(3, 8, 8))
    assert ep.ep_lora_workspace_bytes(lay, 16, 16, 8) > 0
    assert ep.ep_lora_workspace_bytes(lay, 16, 16, 12) == 0
    stale = lay.handle()
    lay.generation += 1
    with pytest.raises(ep.StaleLayoutError):
        ep.ep_lora(z(8, 16), stale, z(3, 8, 16), z(3, 16, 8))
    assert layer.ep_lora is ep.ep_lora


def _geom(T, K, E, H, N, R, A=0, backward=1):
    p, w = _lib.Problem(T, H, K, E, 0, A, 0), _weights(rank=R, n_out=N)
    return _lib.lib().ep_lora_workspace_bytes(ctypes.byref(p), ctypes.byref(w), backward)


def test_workspace_covers_every_split_of_the_rows():
    """The partial weight gradients' bound: experts of several chunks have
    fewer than twice their rows over the chunk size, whatever the split."""
    import random

    rng = random.Random(1)
    for _ in range(300):
        E, rows = rng.randint(1, 40), rng.randint(1, 5000)
        cuts = sorted(rng.randint(0, rows) for _ in range(E - 1))
        counts = [b - a for a, b in zip([0, *cuts], [*cuts, rows])]
        shift = 7
        while shift < 12 and (32 << shift) < rows:
            shift += 1
        chunks = [(c + (1 << shift) - 1) >> shift for c in counts]
        assert sum(c for c in chunks if c > 1) <= 2 * (rows >> shift)
        assert sum(chunks) <= (rows >> shift) + min(rows, E)
        u_and_v = _geom(rows, 1, E, 64, 64, 8, backward=1) - 2 * (rows >> shift) * 8 * 128 * 4
        assert u_and_v >= 2 * rows * 8 * 4


def _parts(rows, E, H, N, R):
    """Bytes of the backward workspace's parts as the kernels index them, for
    H and N below 512 (contractions are not split): 16 a result tile and
    weight-gradient chunk, R fp32 a row of u and of v, R * (H + N) a slot."""
    used, up8 = min(rows, E), lambda n: (n + 7) // 8 * 8
    tile = 7 if R <= 64 else 6
    while tile > 4 and rows >> tile < 192:
        tile -= 1
    chunk = 7
    while chunk < 12 and 32 << chunk < rows:
        chunk += 1
    return tile, chunk, dict(tiles=16 * up8((rows >> tile) + used), chunks=16 * up8((rows >> chunk) + used),
                             u=rows * R * 4, v=rows * R * 4, slots=2 * (rows >> chunk) * R * (H + N) * 4)


@pytest.mark.parametrize("R", [8, 64, 128])
def test_workspace_parts_to_the_byte(R):
    """The library reserves each part in full, at sizes on both sides of every
    step, and each part holds what a split of the rows over experts puts there."""
    import random

    rng = random.Random(R)
    sizes = [1, 2, 127, 128, 129, 4095, 4096, 4097, 8191, 8192, 131_071, 131_072, 131_073, 300_000]
    sizes += [rng.randint(1, 5000) for _ in range(60)] + [rng.randint(5000, 400_000) for _ in range(30)]
    for rows in sizes:
        E, H, N = rng.randint(1, 40), 8 * rng.randint(1, 63), 8 * rng.randint(1, 63)
        tile, chunk, parts = _parts(rows, E, H, N, R)
        assert _geom(rows, 1, E, H, N, R) == sum(parts.values()), (rows, E, H, N, parts)
        for even in (False, True):
            if even:  # every expert just past a whole number of chunks, as far as the rows go
                counts, left = [], rows
                for _ in range(E):
                    n = min(left, ((rows // E >> chunk) << chunk) + 1)
                    counts.append(n)
                    left -= n
                counts[-1] += left
            else:
                cuts = sorted(rng.randint(0, rows) for _ in range(E - 1))
                counts = [b - a for a, b in zip([0, *cuts], [*cuts, rows])]
            assert sum(counts) == rows
            up = lambda c, s: (c + (1 << s) - 1) >> s  # noqa: E731
            many = sum(up(c, chunk) for c in counts if up(c, chunk) > 1)
            assert 16 * sum(up(c, tile) for c in counts) <= parts["tiles"]
            assert 16 * sum(up(c, chunk) for c in counts) <= parts["chunks"]
            assert many * R * (H + N) * 4 <= parts["slots"]
    # padding to an alignment takes rows too
    assert _geom(100, 2, 8, 64, 64, R, A=16) == sum(_parts(200 + 8 * 15, 8, 64, 64, R)[2].values())
