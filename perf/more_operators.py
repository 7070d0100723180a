"""The experts' layers and the router's balance loss, as cases that can be
timed and compared.

``ep_expert_linear`` is an expert's layer over the layout's segments: the
grouped product with bias, activation (gated or not) and residual in its
epilogue; ``ep_expert_linear_backward`` is its gradient to the rows, the
weights and the bias.  ``ep_balance_loss`` counts each expert's selections and
weighs them with the router's mean scores, sequence by sequence, and
``ep_balance_loss_backward`` takes it to the logits.

``run`` computes them in plain torch operations in 32 bits, or through the
package's entry points where ``own`` is true.  ``exact`` gives the same from
the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

NEG_INF = float("-inf")
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest layer: 128 tokens x 256, top-2 of 16.  Latency counts.
        dict(name="linear tiny", op="linear", T=128, E=16, K=2, H=256, N=256, act="gelu", gated=False, bias=True,
             residual=True, gather=False, pre=False, masked=0.1, zipf=0.0),
        # One decoding step of 16 sequences through the mid-sized layer's gated
        # projection: a row or two an expert, the weights are what is read.
        dict(name="linear decode", op="linear", T=16, E=64, K=4, H=4096, N=2048, act="silu", gated=True, bias=False,
             residual=False, gather=True, pre=False, masked=0.0, zipf=0.0),
        # The same projection over a training batch: the dispatch is folded
        # into the loads, the values before the activation are kept.
        dict(name="linear gated mid", op="linear", T=4096, E=64, K=4, H=4096, N=2048, act="silu", gated=True,
             bias=False, residual=False, gather=True, pre=True, masked=0.0, zipf=0.0),
        # The way back down, uneven experts and odd sizes, bias and residual.
        dict(name="linear down odd", op="linear", T=4093, E=61, K=3, H=2008, N=4104, act="none", gated=False,
             bias=True, residual=True, gather=False, pre=False, masked=0.05, zipf=0.25),
        # The full layer: 8192 tokens x 7168, top-8 of 256 experts.
        dict(name="linear full", op="linear", T=8192, E=256, K=8, H=7168, N=2048, act="gelu_tanh", gated=False,
             bias=True, residual=False, gather=False, pre=False, masked=0.0, zipf=0.0),
        # A small fine-tuning batch on odd sizes.
        dict(name="linear backward small", op="linear_backward", T=509, E=8, K=2, H=1032, N=520, act="gelu",
             gated=False, bias=True, gather=True, masked=0.1, zipf=0.0),
        # The gradient of the mid-sized layer's gated projection.
        dict(name="linear backward gated mid", op="linear_backward", T=4096, E=64, K=4, H=4096, N=2048, act="silu",
             gated=True, bias=False, gather=True, masked=0.0, zipf=0.0),
        # One rank's share of the full layer: 32 experts of about 2048 rows.
        dict(name="linear backward rank", op="linear_backward", T=8192, E=32, K=8, H=7168, N=2048, act="none",
             gated=False, bias=True, gather=False, masked=0.0, zipf=0.25),
        # A fine-tuning batch of ragged sequences, a part of it padding.
        dict(name="balance small", op="balance", T=509, E=64, K=4, score="softmax", dtype="fp32", B=7, masked=0.1,
             tail=13),
        # The receive share of a whole node: balanced within each sequence.
        dict(name="balance large", op="balance", T=65536, E=256, K=8, score="sigmoid", dtype="fp32", B=16, masked=0.02,
             tail=0),
        # The gradient over one rank's batch as a whole.
        dict(name="balance backward mid", op="balance_backward", T=8192, E=256, K=8, score="softmax", dtype="bf16", B=0,
             masked=0.02, tail=0, base=False),
        # And over the large batch, added to the gradient that came through
        # the weights.
        dict(name="balance backward large", op="balance_backward", T=65536, E=256, K=8, score="sigmoid", dtype="fp32",
             B=16, masked=0.02, tail=100, base=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "balance", "balance_backward"])
    if op in ("balance", "balance_backward"):
        T, E = _log_int(rng, 1, 60000), rng.randint(4, 320)
        B = rng.choice([0, 0, _log_int(rng, 1, 300)])
        c = dict(op=op, T=T, E=E, K=rng.randint(1, min(10, E)), score=rng.choice(["softmax", "sigmoid"]),
                 dtype=rng.choice(["fp32", "bf16"]), B=B, masked=rng.choice([0.0, 0.05]),
                 tail=rng.randint(0, T // 8) if B else 0)
        if op == "balance_backward":
            c["base"] = rng.random() < 0.5
        return c
    E = rng.randint(1, 64)
    K = rng.randint(1, min(4, E))
    gated = rng.random() < 0.4
    c = dict(op=op, T=_log_int(rng, 1, 4096), E=E, K=K, H=8 * _log_int(rng, 8, 512),
             N=8 * _log_int(rng, 8, 256 if gated else 512), act=rng.choice(ACTS), gated=gated, bias=rng.random() < 0.5,
             gather=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]), zipf=rng.choice([0.0, 0.5]))
    if op == "linear":
        c.update(residual=rng.random() < 0.5, pre=rng.random() < 0.5)
    return c


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32)


def _bf(g, scale, *shape):
    return (_randn(g, *shape) * scale).to(torch.bfloat16)


def _pick(g, T, K, E, zipf):
    """K distinct of E per token (Gumbel top-K over popularity rank^-zipf)."""
    logp = -zipf * torch.log(torch.arange(1, E + 1, device=_dev(), dtype=torch.float32))
    logp = logp[torch.randperm(E, generator=g, device=_dev())]
    u = torch.rand(T, E, generator=g, device=_dev()).clamp_(min=1e-20)
    return (logp - torch.log((-torch.log(u)).clamp_(min=1e-20))).topk(K, dim=1).indices


def _segments(ids, E, K):
    """The expert-major order of the flat selections ids [T*K] (-1: none):
    source token of each row, rows per expert, and for each expert its rows
    padded to the longest segment."""
    key = torch.where(ids < 0, torch.full_like(ids, E), ids)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    rows = int(counts.sum())
    offsets = torch.cumsum(counts, 0) - counts
    width = max(1, int(counts.max()))
    at = torch.arange(width, device=ids.device)
    valid = at < counts[:, None]
    padded = torch.where(valid, offsets[:, None] + at, 0)
    return dict(src=order[:rows] // K, counts=counts, rows=rows, padded=padded, valid=valid)


def _prepare_linear(s, c, g):
    T, E, K, H, N = (c[k] for k in "TEKHN")
    wide = 2 * N if c["gated"] else N
    ids = _pick(g, T, K, E, c["zipf"])
    if c["masked"]:
        ids = torch.where(torch.rand(T, K, generator=g, device=_dev()) < c["masked"], -1, ids)
    ids = ids.contiguous()
    seg = _segments(ids.reshape(-1), E, K)
    rows = T * K
    w = torch.empty(E, wide, H, dtype=torch.bfloat16, device=_dev())
    for e in range(E):  # one expert at a time keeps the 32-bit temporary small
        w[e] = _bf(g, H**-0.5, wide, H)
    s.update(seg=seg, w=w, x=_bf(g, 1.0, T if c["gather"] else rows, H),
             b=_bf(g, 0.5, E, wide) if c["bias"] else None)
    # the row of x that each expert-major row is
    s["at"] = seg["src"] if c["gather"] else torch.arange(seg["rows"], device=_dev())
    bare = c["act"] == "none" and not c["gated"]
    if c["op"] == "linear":
        s["res"] = _bf(g, 1.0, rows, N) if c["residual"] else None
        s["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=_dev())
        s["pre"] = torch.zeros(rows, wide, dtype=torch.bfloat16, device=_dev()) if c["pre"] else None
    else:
        s["go"] = _bf(g, 1e-2, rows, N)
        s["pre"] = None if bare else _bf(g, 1.0, rows, wide)
        s["gpre"] = None if bare else torch.zeros(rows, wide, dtype=torch.bfloat16, device=_dev())
        s["gx"] = torch.zeros(rows, H, dtype=torch.bfloat16, device=_dev())
    if own:
        import combine_ep_layout_03_amd as ep

        # placed once for a batch; every product of the layer uses it
        s["layout"] = ep.ep_layout(ids, E, expert_row_src=True)


def _prepare_balance(s, c, g):
    T, E, K, B = (c[k] for k in "TEKB")
    # a router in training: tokens spread over experts of uneven popularity
    logits = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
    s["logits"] = logits if c["dtype"] == "fp32" else logits.to(torch.bfloat16)
    s["mask"] = torch.rand(T, generator=g, device=_dev()) >= c["masked"] if c["masked"] else None
    idx = logits.topk(K, dim=1).indices
    s["idx"] = (idx if s["mask"] is None else torch.where(s["mask"][:, None], idx, -1)).contiguous()
    if B:
        # ragged sequences, the last of them ending `tail` tokens early
        end = T - c["tail"]
        cuts = torch.sort(torch.randint(0, end + 1, (B - 1,), generator=g, device=_dev())).values
        zero = torch.zeros(1, dtype=torch.int64, device=_dev())
        s["seq"] = torch.cat([zero, cuts, zero + end]).to(torch.int32)
    else:
        s["seq"] = None
    if c["op"] == "balance_backward":
        s["gl"] = _randn(g, 1).abs() + 0.5
        base = 1e-6 * _randn(g, T, E) if c["base"] else None
        s["base"] = base if base is None or c["dtype"] == "fp32" else base.to(torch.bfloat16)
        s["counts"], s["tokens"] = _counts(s)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("linear", "linear_backward"):
        _prepare_linear(s, case, g)
    else:
        _prepare_balance(s, case, g)
    return s


# ------------------------------------------------------------ plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _padded(t, at, s):
    """Rows `at` of t by expert, [E, longest, width] in 32 bits, zero past a
    segment's end."""
    seg = s["seg"]
    if seg["rows"] == 0:
        return torch.zeros(*seg["padded"].shape, t.shape[1], device=t.device)
    return torch.where(seg["valid"][:, :, None], t[at[seg["padded"]]].float(), 0.0)


def _own_rows(s):
    return torch.arange(s["seg"]["rows"], device=_dev())


def _placed(v, rows, s):
    """Expert-major rows v [E, longest, width] as bf16 [rows, width], zero
    where no selection is."""
    seg = s["seg"]
    out = torch.zeros(rows, v.shape[2], dtype=torch.bfloat16, device=v.device)
    out[: seg["rows"]] = v[seg["valid"]].to(torch.bfloat16)
    return out


def _plain_linear(s):
    c = s["case"]
    N, rows = c["N"], c["T"] * c["K"]
    # [E, wide, longest]: the weights as they lie, the rows turned
    x = _padded(s["x"], s["at"], s).transpose(1, 2).contiguous()
    z = torch.bmm(s["w"].float(), x).transpose(1, 2)
    if s["b"] is not None:
        z = z + s["b"].float()[:, None, :]
    y = _act(z[:, :, :N], c["act"]) * z[:, :, N:] if c["gated"] else _act(z, c["act"])
    if s["res"] is not None:
        y = y + _padded(s["res"], _own_rows(s), s)
    out = _placed(y, rows, s)
    return (out, _placed(z, rows, s)) if c["pre"] else (out,)


def _plain_linear_backward(s):
    c = s["case"]
    N, rows = c["N"], c["T"] * c["K"]
    g = _padded(s["go"], _own_rows(s), s)
    if s["pre"] is not None:
        z = _padded(s["pre"], _own_rows(s), s)
        if c["gated"]:
            a, b = z[:, :, :N], z[:, :, N:]
            g = torch.cat([g * b * _slope(a, c["act"]), g * _act(a, c["act"])], 2)
        else:
            g = g * _slope(z, c["act"])
    x = _padded(s["x"], s["at"], s)
    gx = _placed(torch.bmm(g, s["w"].float()), rows, s)
    gw = torch.bmm(g.transpose(1, 2), x).to(torch.bfloat16)
    out = [gx, gw]
    if s["b"] is not None:
        out.append(g.sum(1).to(torch.bfloat16))
    if s["pre"] is not None:
        out.append(_placed(g, rows, s))
    return out


def _sequence_of(s):
    """Sequence of each token, B for the tokens of none, and B."""
    T = s["case"]["T"]
    if s["seq"] is None:
        return torch.zeros(T, dtype=torch.int64, device=_dev()), 1
    B = s["seq"].numel() - 1
    at = torch.arange(T, device=_dev())
    return torch.searchsorted(s["seq"][1:].long().contiguous(), at, right=True).clamp(max=B), B


def _counts(s):
    """Selections of each expert [B, E] and tokens [B] of each sequence."""
    c = s["case"]
    E = c["E"]
    seq, B = _sequence_of(s)
    live = torch.ones_like(seq, dtype=torch.bool) if s["mask"] is None else s["mask"]
    seq = torch.where(live, seq, B)
    tokens = torch.bincount(seq, minlength=B + 1)[:B].to(torch.int32)
    key = torch.where(s["idx"] < 0, B * E, seq[:, None] * E + s["idx"]).clamp(max=B * E)
    counts = torch.bincount(key.reshape(-1), minlength=B * E + 1)[: B * E].reshape(B, E).to(torch.int32)
    return counts, tokens


def _mean_scores(l, score):
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
    else:
        e = 1.0 / (1.0 + torch.exp(-l))
    return e / e.sum(1, keepdim=True)


COEF = 1e-2


def _plain_balance(s):
    c = s["case"]
    counts, tokens = _counts(s)
    seq, B = _sequence_of(s)
    p = _mean_scores(s["logits"].float(), c["score"])
    if s["mask"] is not None:
        p = torch.where(s["mask"][:, None], p, 0.0)
    # long sums: in 64 bits
    member = seq == torch.arange(B, device=p.device)[:, None]
    n = tokens.double().clamp(min=1.0)[:, None]
    mean = (member.double() @ p.double()) / n
    loss = COEF * c["E"] / (c["K"] * B) * (counts.double() / n * mean).sum()
    return loss.float().reshape(1), counts, tokens, mean.float()


def _plain_balance_backward(s):
    c = s["case"]
    seq, B = _sequence_of(s)
    l = s["logits"].float()
    p = _mean_scores(l, c["score"])
    n = s["tokens"].float().clamp(min=1.0)
    f = s["counts"].float() * (COEF * c["E"] / (c["K"] * B) / (n * n))[:, None] * s["gl"]
    f = torch.cat([f, torch.zeros_like(f[:1])])[seq]
    if s["mask"] is not None:
        f = torch.where(s["mask"][:, None], f, 0.0)
    d = p * (f - (f * p).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(l))
    if s["base"] is not None:
        d = d + s["base"].float()
    return d.to(s["logits"].dtype)


# -------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "balance": _plain_balance,
                "balance_backward": _plain_balance_backward}[op](s)
    import combine_ep_layout_03_amd as ep

    if op == "linear":
        out = ep.ep_expert_linear(s["x"], s["layout"], s["w"], bias=s["b"], activation=_activation(ep, c),
                                  gated=c["gated"], residual=s["res"], gather=c["gather"], out=s["out"], pre=s["pre"])
        return (out, s["pre"]) if c["pre"] else (out,)
    if op == "linear_backward":
        gx, gw, gb, gpre = ep.ep_expert_linear_backward(
            s["go"], s["x"], s["layout"], s["w"], pre=s["pre"], activation=_activation(ep, c), gated=c["gated"],
            gather=c["gather"], bias=c["bias"], grad_x=s["gx"], grad_pre=s["gpre"])
        return [gx, gw] + ([gb] if c["bias"] else []) + ([] if s["pre"] is None else [gpre])
    if op == "balance":
        return ep.ep_balance_loss(s["logits"], s["idx"], score=_score(ep, c), coef=COEF, seq_offsets=s["seq"],
                                  token_mask=s["mask"])
    return ep.ep_balance_loss_backward(s["gl"], s["logits"], s["counts"], s["tokens"], c["K"], score=_score(ep, c),
                                       coef=COEF, seq_offsets=s["seq"], token_mask=s["mask"], grad_base=s["base"])


def _activation(ep, c):
    return {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU,
            "gelu_tanh": ep.EP_ACT_GELU_TANH}[c["act"]]


def _score(ep, c):
    return ep.EP_SCORE_SIGMOID if c["score"] == "sigmoid" else ep.EP_SCORE_SOFTMAX


# ------------------------------------------------------------------- work
def work(case):
    op, T, E, K = case["op"], case["T"], case["E"], case["K"]
    if op in ("balance", "balance_backward"):
        el, B = 4 if case["dtype"] == "fp32" else 2, max(1, case["B"])
        if op == "balance":
            return {"bytes": T * E * el + T * K * 8 + 8 * B * E, "flops": 4 * T * E}
        return {"bytes": (3 if case["base"] else 2) * T * E * el + 4 * B * E, "flops": 6 * T * E}
    H, N = case["H"], case["N"]
    wide = 2 * N if case["gated"] else N
    n = T * K * (1 - case["masked"])
    xrows = min(T, n) if case["gather"] else n
    # experts that get a row, if all were equally likely
    used = E * (1 - (1 - 1 / E) ** n) if n else 0
    if op == "linear":
        more = (N if case["residual"] else 0) + (wide if case["pre"] else 0)
        return {"bytes": 2 * (used * wide * H + xrows * H + n * N + n * more), "flops": 2 * n * wide * H}
    bare = case["act"] == "none" and not case["gated"]
    return {"bytes": 2 * (used * wide * H + E * wide * H + xrows * H + n * H + n * N + (0 if bare else 2 * n * wide)),
            "flops": 4 * n * wide * H}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "linear_backward": _exact_linear_backward, "balance": _exact_balance,
            "balance_backward": _exact_balance_backward}[case["op"]](s, case)


def _act64(z, act):
    """(activation, its derivative) of float64 z."""
    if act == "relu":
        on = (z > 0).double()
        return z * on, on
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        a = (2 / math.pi) ** 0.5
        u = a * z + a * 0.044715 * z**3
        p = torch.sigmoid(2 * u)  # (1 + tanh u) / 2
        return z * p, p + z * 2 * p * (1 - p) * (a + 3 * a * 0.044715 * z**2)
    return z, torch.ones_like(z)


def _each_expert(s):
    """(expert, its rows of x, its first row, one past its last)."""
    r0 = 0
    for e, n in enumerate(s["seg"]["counts"].tolist()):
        if n:
            yield e, s["at"][r0:r0 + n], r0, r0 + n
        r0 += n


def _exact_linear(s, c):
    N = c["N"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=_dev())
    pre = torch.zeros(s["pre"].shape, dtype=torch.float64, device=_dev()) if c["pre"] else None
    for e, at, r0, r1 in _each_expert(s):
        z = s["x"][at].double() @ s["w"][e].double().T
        if s["b"] is not None:
            z += s["b"][e].double()
        y = _act64(z[:, :N], c["act"])[0]
        if c["gated"]:
            y = y * z[:, N:]
        if s["res"] is not None:
            y = y + s["res"][r0:r1].double()
        out[r0:r1] = y
        if c["pre"]:
            pre[r0:r1] = z
    return (out, pre) if c["pre"] else (out,)


def _exact_linear_backward(s, c):
    N = c["N"]
    gx = torch.zeros(s["gx"].shape, dtype=torch.float64, device=_dev())
    gw = torch.zeros(s["w"].shape, dtype=torch.float64, device=_dev())
    gb = torch.zeros(s["w"].shape[:2], dtype=torch.float64, device=_dev())
    gz = None if s["pre"] is None else torch.zeros(s["pre"].shape, dtype=torch.float64, device=_dev())
    for e, at, r0, r1 in _each_expert(s):
        g = s["go"][r0:r1].double()
        if gz is not None:
            z = s["pre"][r0:r1].double()
            value, slope = _act64(z[:, :N], c["act"])
            g = torch.cat([g * slope * z[:, N:], g * value], 1) if c["gated"] else g * slope
            gz[r0:r1] = g
        gx[r0:r1] = g @ s["w"][e].double()
        gw[e] = g.T @ s["x"][at].double()
        gb[e] = g.sum(0)
    return [gx, gw] + ([gb] if s["b"] is not None else []) + ([gz] if gz is not None else [])


def _sequences(s, c):
    """(sequence, its live tokens) by their offsets."""
    off = [0, c["T"]] if s["seq"] is None else s["seq"].tolist()
    mask = np.ones(c["T"], bool) if s["mask"] is None else s["mask"].cpu().numpy()
    for b in range(len(off) - 1):
        at = np.arange(off[b], off[b + 1])
        yield b, at[mask[at]]


def _share64(s, c):
    l = s["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        e = np.exp(l - l.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True), np.ones_like(l)
    e = 1 / (1 + np.exp(-l))
    return e / e.sum(1, keepdims=True), 1 / (1 + np.exp(l))


def _exact_balance(s, c):
    E, K = c["E"], c["K"]
    p, _ = _share64(s, c)
    idx = s["idx"].cpu().numpy()
    B = 1 if s["seq"] is None else s["seq"].numel() - 1
    loss, counts, tokens, mean = 0.0, np.zeros((B, E), np.int32), np.zeros(B, np.int32), np.zeros((B, E))
    for b, at in _sequences(s, c):
        tokens[b] = len(at)
        chosen = idx[at]
        counts[b] = np.bincount(chosen[chosen >= 0].reshape(-1), minlength=E)
        if len(at):
            mean[b] = p[at].mean(0)
            loss += COEF / B * (E / (K * len(at)) * counts[b] * mean[b]).sum()
    return torch.tensor([loss], dtype=torch.float64), torch.from_numpy(counts), torch.from_numpy(tokens), \
        torch.from_numpy(mean)


def _exact_balance_backward(s, c):
    E, K = c["E"], c["K"]
    p, rest = _share64(s, c)
    counts = s["counts"].cpu().numpy().astype(np.float64)
    g = float(s["gl"].double())
    d = np.zeros_like(p)
    for b, at in _sequences(s, c):
        if len(at):
            # d loss / d mean share of each token, then through the share
            f = g * COEF / counts.shape[0] * E / (K * len(at)) * counts[b] / len(at)
            q = p[at]
            d[at] = q * rest[at] * (f - (q * f).sum(1, keepdims=True))
    d = torch.from_numpy(d)
    return d if s["base"] is None else d + s["base"].double().cpu()
