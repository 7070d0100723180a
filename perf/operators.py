"""The operators around dispatch and combine, as cases that can be timed and compared.

Routing (``ep_route``) makes the selections that the layout places; the
gradient of the combine (``ep_combine_backward``) brings back each expert
row's gradient and each selection weight's, and ``ep_route_backward`` takes
the latter to the logits; ``ep_lora`` adds low-rank adapters beside a shared
or an expert's projection over the layout's segments, and
``ep_lora_backward`` is its gradient.

``run`` computes them in plain torch operations in 32 bits (selections in 64,
where neighbouring scores decide), or through the package's entry points
where ``own`` is true.  ``exact`` gives the same from the definitions in 64
bits.
"""
import math

import numpy as np
import torch

own = False

NEG_INF = float("-inf")


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of 16 sequences: sigmoid scores, balance bias, 4 of
        # 8 expert groups, renormalised.  Latency is all that counts.
        dict(name="route decode", op="route", T=16, E=256, K=8, score="sigmoid", bias=True, G=8, TG=4, gtop=2,
             renorm=True, scale=2.5, dtype="fp32", masked=0.0, drained=0),
        # The same router over one rank's prefill batch, a part of it padding
        # and two experts drained (their logits are -inf).
        dict(name="route prefill", op="route", T=8192, E=256, K=8, score="sigmoid", bias=True, G=8, TG=4, gtop=2,
             renorm=True, scale=2.5, dtype="fp32", masked=0.02, drained=2),
        # The receive share of a whole node at once: plain softmax routing on
        # bf16 logits, where equal logits are common.
        dict(name="route large", op="route", T=65536, E=256, K=8, score="softmax", bias=False, G=0, TG=0, gtop=1,
             renorm=True, scale=1.0, dtype="bf16", masked=0.0, drained=0),
        # A training step of the mid-sized layer: softmax over all experts, not
        # renormalised, so the gradient of a row is dense.
        dict(name="route backward mid", op="route_backward", T=4096, E=64, K=4, score="softmax", bias=False, G=0,
             TG=0, gtop=1, renorm=False, scale=1.0, dtype="fp32", masked=0.0, drained=0),
        # Training at the large batch: sigmoid, renormalised (a sparse row).
        dict(name="route backward large", op="route_backward", T=65536, E=256, K=8, score="sigmoid", bias=True, G=8,
             TG=4, gtop=2, renorm=True, scale=2.5, dtype="fp32", masked=0.02, drained=0),
        # The smallest workload: gradient of 128 tokens x 256.
        dict(name="combine backward tiny", op="combine_backward", T=128, H=256, K=2, E=16, zipf=0.0, masked=0.1),
        # The full layer: 8192 tokens x 7168, top-8 of 256.
        dict(name="combine backward full", op="combine_backward", T=8192, H=7168, K=8, E=256, zipf=0.0, masked=0.0),
        # One new token for each of 61 sequences, most with an adapter of
        # their own, beside a 4096 x 4096 projection.
        dict(name="lora decode", op="lora", T=61, E=48, K=1, H=4096, N=4096, R=16, rows="tokens", requests=61,
             none=0.1, zipf=0.0),
        # Prompts of 23 requests of uneven length, 12 adapters, rank 64,
        # beside a projection 7168 -> 2048.
        dict(name="lora prefill", op="lora", T=8111, E=12, K=1, H=7168, N=2048, R=64, rows="tokens", requests=23,
             none=0.1, zipf=1.0),
        # An adapter for each expert over the dispatched rows of the mid-sized
        # layer (4096 tokens, top-4 of 64), beside the grouped GEMM.
        dict(name="lora experts", op="lora", T=4096, E=64, K=4, H=4096, N=2048, R=32, rows="experts", requests=0,
             none=0.05, zipf=0.5),
        # A small fine-tuning batch of 4 adapters at once.
        dict(name="lora backward small", op="lora_backward", T=509, E=4, K=1, H=4096, N=4096, R=8, rows="tokens",
             requests=9, none=0.0, zipf=0.0),
        # Adapters of the experts trained over the dispatched rows of the
        # mid-sized layer.
        dict(name="lora backward experts", op="lora_backward", T=4096, E=64, K=4, H=4096, N=2048, R=32,
             rows="experts", requests=0, none=0.05, zipf=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "lora", "lora_backward"])
    if op in ("route", "route_backward"):
        G = rng.choice([0, 0, 2, 4, 8])
        E = rng.randint(4, 40) * G if G else rng.randint(8, 320)
        TG = rng.randint(1, G) if G else 0
        K = rng.randint(1, min(10, E * TG // G if G else E))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log_int(rng, 1, 40000), E=E, K=K, score=score, bias=rng.random() < 0.5, G=G, TG=TG,
                    gtop=rng.choice([1, 2]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["fp32", "bf16"]), masked=rng.choice([0.0, 0.05]), drained=rng.choice([0, 1]))
    if op == "combine_backward":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log_int(rng, 1, 6000), H=_log_int(rng, 100, 7168), K=rng.randint(1, 8), E=E,
                    zipf=rng.choice([0.0, 1.2]), masked=rng.choice([0.0, 0.1]))
    rows = rng.choice(["tokens", "experts"])
    H, N = 8 * _log_int(rng, 16, 896), 8 * _log_int(rng, 16, 512)
    R = rng.choice([8, 16, 24, 32, 40, 64, 128])
    if rows == "tokens":
        T, E, K, req = _log_int(rng, 1, 6000), rng.randint(1, 48), 1, rng.randint(1, 64)
    else:
        T, E, K, req = _log_int(rng, 1, 2000), rng.randint(8, 64), rng.randint(1, 4), 0
    return dict(op=op, T=T, E=E, K=K, H=H, N=N, R=R, rows=rows, requests=min(req, T), none=rng.choice([0.0, 0.1]),
                zipf=rng.choice([0.0, 1.0]))


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32)


def _pick(g, T, K, E, zipf):
    """K distinct of E per token (Gumbel top-K over popularity rank^-zipf)."""
    logp = -zipf * torch.log(torch.arange(1, E + 1, device=_dev(), dtype=torch.float32))
    logp = logp[torch.randperm(E, generator=g, device=_dev())]
    u = torch.rand(T, E, generator=g, device=_dev()).clamp_(min=1e-20)
    return (logp - torch.log(-torch.log(u).clamp_(min=1e-20))).topk(K, dim=1).indices


def _segments(ids, E, K):
    """The expert-major order of the flat selections ids [T*K] (-1: none):
    slot per selection, source token per row, rows per expert, and for each
    expert its rows padded to the longest segment."""
    n = ids.numel()
    key = torch.where(ids < 0, torch.full_like(ids, E), ids)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    rows = int(counts.sum())
    slot = torch.full((n,), -1, dtype=torch.int64, device=ids.device)
    slot[order[:rows]] = torch.arange(rows, device=ids.device)
    src = order[:rows] // K
    offsets = torch.cumsum(counts, 0) - counts
    width = max(1, int(counts.max()))
    at = torch.arange(width, device=ids.device)
    valid = at < counts[:, None]
    padded = torch.where(valid, offsets[:, None] + at, 0)
    return dict(slot=slot, src=src, counts=counts, rows=rows, padded=padded, valid=valid)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        # a trained router: tokens spread over experts of uneven popularity
        logits = 1.5 * _randn(g, T, E) + 0.3 * _randn(g, E)
        if case["drained"]:
            logits[:, torch.randperm(E, generator=g, device=_dev())[: case["drained"]]] = NEG_INF
        s["logits"] = logits if case["dtype"] == "fp32" else logits.to(torch.bfloat16)
        # the balance bias moves by fixed steps
        s["bias"] = (_randn(g, E) * 40).round() * 1e-3 if case["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device=_dev()) >= case["masked"] if case["masked"] else None
        if op == "route_backward":
            s["idx"] = _plain_route(s)[0]
            s["gw"] = _randn(g, T, K)
    elif op == "combine_backward":
        T, H, K, E = case["T"], case["H"], case["K"], case["E"]
        ids = _pick(g, T, K, E, case["zipf"])
        if case["masked"]:
            ids = torch.where(torch.rand(T, K, generator=g, device=_dev()) < case["masked"], -1, ids)
        ids = ids.contiguous()
        seg = _segments(ids.reshape(-1), E, K)
        s["slot"] = seg["slot"].reshape(T, K)
        s["w"] = torch.softmax(_randn(g, T, K), 1)
        s["y"] = _randn(g, T * K, H).to(torch.bfloat16)
        s["go"] = (_randn(g, T, H) * 1e-2).to(torch.bfloat16)
        s["gy"] = torch.zeros(T * K, H, dtype=torch.bfloat16, device=_dev())
        if own:
            import combine_ep_layout_03_amd as ep

            s["layout"] = ep.ep_layout(ids, E)
    else:
        T, E, K, H, N, R = (case[k] for k in "TEKHNR")
        if case["rows"] == "tokens":
            # whole requests, each with one adapter or none
            q = case["requests"]
            who = _pick(g, q, 1, E, case["zipf"]).reshape(-1)
            who = torch.where(torch.rand(q, generator=g, device=_dev()) < case["none"], -1, who)
            cuts = torch.sort(torch.randperm(T - 1, generator=g, device=_dev())[: q - 1] + 1).values if q > 1 else None
            starts = torch.zeros(T, dtype=torch.int64, device=_dev())
            if cuts is not None:
                starts[cuts] = 1
            ids = who[torch.cumsum(starts, 0)].reshape(T, 1).contiguous()
            xrows = T
        else:
            ids = _pick(g, T, K, E, case["zipf"])
            ids = torch.where(torch.rand(T, K, generator=g, device=_dev()) < case["none"], -1, ids).contiguous()
            xrows = T * K
        seg = _segments(ids.reshape(-1), E, K)
        s.update(seg=seg, x=_randn(g, xrows, H).to(torch.bfloat16),
                 a=(_randn(g, E, R, H) * H**-0.5).to(torch.bfloat16),
                 b=(_randn(g, E, N, R) * R**-0.5).to(torch.bfloat16),
                 scales=torch.rand(E, generator=g, device=_dev()) + 0.5)
        # the row of x, base and out that each expert-major row is
        s["at"] = seg["src"] if case["rows"] == "tokens" else torch.arange(seg["rows"], device=_dev())
        if op == "lora":
            s["base"] = _randn(g, xrows, N).to(torch.bfloat16)
            s["out"] = torch.zeros(xrows, N, dtype=torch.bfloat16, device=_dev())
        else:
            s["go"] = (_randn(g, xrows, N) * 1e-2).to(torch.bfloat16)
            s["gx"] = torch.zeros(xrows, H, dtype=torch.bfloat16, device=_dev())
        if own:
            import combine_ep_layout_03_amd as ep

            # placed once for a batch; every projection of every layer uses it
            s["layout"] = ep.ep_layout(ids, E, expert_row_src=True)
    return s


# ------------------------------------------------------------ plain forms
def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e300))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _chosen_weights(l, sel, score, renorm):
    """Scores of the selected logits l [T, K] (sel: which are selections)
    divided by their sum, stable where all of them are tiny."""
    top = torch.where(sel, l, NEG_INF).amax(1, keepdim=True)
    top = torch.where(top == NEG_INF, 0.0, top)
    if score == "softmax":
        e = torch.exp(l - top)
    else:
        # sigmoid(l) = exp(-log(1 + exp(-l))), relative to the largest
        logs = torch.clamp(l, max=0.0) - torch.log1p(torch.exp(-l.abs()))
        ltop = torch.clamp(top, max=0.0) - torch.log1p(torch.exp(-top.abs()))
        e = torch.exp(logs - ltop)
    e = torch.where(sel, e, 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-37)


def _plain_route(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    logits, bias = s["logits"], s["bias"]
    # neighbouring scores decide: the selection is made in 64 bits
    l64 = logits.double()
    bad = logits == NEG_INF
    if bias is None:
        key = l64  # both scores grow with the logit
    else:
        key = _scores(l64, c["score"]) + bias.double()
    key = torch.where(bad, NEG_INF, key)
    if G:
        per = key if bias is not None or c["gtop"] == 1 else torch.where(bad, NEG_INF, _scores(l64, c["score"]))
        best = torch.sort(per.reshape(T, G, E // G), dim=2, descending=True).values[:, :, : min(c["gtop"], E // G)]
        gs = torch.where(best == NEG_INF, 0.0, best).sum(2)
        gs = torch.where(best[:, :, 0] == NEG_INF, NEG_INF, gs)
        keep = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, : c["TG"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, keep, True)
        key = torch.where(open_.repeat_interleave(E // G, 1), key, NEG_INF)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    idx, sel = order.indices[:, :K], order.values[:, :K] > NEG_INF
    if s["mask"] is not None:
        sel = sel & s["mask"][:, None]
    l = logits.float()
    if c["renorm"]:
        w = _chosen_weights(torch.gather(l, 1, idx), sel, c["score"], True)
    elif c["score"] == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(-torch.gather(l, 1, idx)))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        w = torch.gather(e, 1, idx) / e.sum(1, keepdim=True)
    return torch.where(sel, idx, -1), torch.where(sel, w * c["scale"], 0.0)


def _plain_route_backward(s):
    c = s["case"]
    l, idx = s["logits"].float(), s["idx"]
    sel = idx >= 0
    at = idx.clamp(min=0)
    gw = torch.where(sel, s["gw"] * c["scale"], 0.0)
    ls = torch.gather(l, 1, at)
    out = torch.zeros_like(l)
    if c["renorm"]:
        w = _chosen_weights(ls, sel, c["score"], True)
        d = w * (gw - (w * gw).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d / (1.0 + torch.exp(ls))
        out.scatter_add_(1, at, torch.where(sel, d, 0.0))
    elif c["score"] == "sigmoid":
        d = gw / (1.0 + torch.exp(ls)) / (1.0 + torch.exp(-ls))
        out.scatter_add_(1, at, torch.where(sel, d, 0.0))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        out.scatter_add_(1, at, gw)
        dot = (torch.gather(p, 1, at) * gw).sum(1, keepdim=True)
        out = p * (out - dot)
    return out.to(s["logits"].dtype)


def _plain_combine_backward(s):
    slot, w, y, go = s["slot"], s["w"], s["y"], s["go"]
    sel = slot >= 0
    at = slot.clamp(min=0)
    g32 = go.float()
    gw = (y[at].float() * g32[:, None, :]).sum(2)
    gy = torch.zeros(y.shape, dtype=torch.bfloat16, device=y.device)
    gy[slot[sel]] = (w[:, :, None] * g32[:, None, :]).to(torch.bfloat16)[sel]
    return gy, torch.where(sel, gw, 0.0)


def _padded(t, s):
    """Rows of t by expert, [E, longest, width] in 32 bits, zero past a
    segment's end."""
    seg = s["seg"]
    if seg["rows"] == 0:
        return torch.zeros(*seg["padded"].shape, t.shape[1], device=t.device)
    return torch.where(seg["valid"][:, :, None], t[s["at"][seg["padded"]]].float(), 0.0)


def _scattered(v, base, s):
    """base (32 bits) with expert-major rows v [E, longest, width] added."""
    seg = s["seg"]
    if seg["rows"]:
        at = s["at"][seg["padded"][seg["valid"]]]
        base[at] += v[seg["valid"]]
    return base


def _plain_lora(s):
    seg = s["seg"]
    u = torch.bmm(_padded(s["x"], s), s["a"].float().transpose(1, 2).contiguous())
    d = torch.bmm(u, s["b"].float().transpose(1, 2).contiguous()) * s["scales"][:, None, None]
    out = s["base"].float()
    if s["case"]["rows"] == "experts":
        out[seg["rows"]:] = 0.0  # rows of no expert are not written
    return _scattered(d, out, s).to(torch.bfloat16)


def _plain_lora_backward(s):
    x, g, sc = _padded(s["x"], s), _padded(s["go"], s), s["scales"][:, None, None]
    a, b = s["a"].float(), s["b"].float()
    u = torch.bmm(x, a.transpose(1, 2).contiguous())
    v = torch.bmm(g, b) * sc
    gx = _scattered(torch.bmm(v, a), torch.zeros_like(s["gx"], dtype=torch.float32), s)
    ga = torch.bmm(v.transpose(1, 2).contiguous(), x)
    gb = torch.bmm(g.transpose(1, 2).contiguous(), u) * sc
    return gx.to(torch.bfloat16), ga.to(torch.bfloat16), gb.to(torch.bfloat16)


# -------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"route": _plain_route, "route_backward": _plain_route_backward,
                "combine_backward": _plain_combine_backward, "lora": _plain_lora,
                "lora_backward": _plain_lora_backward}[op](s)
    import combine_ep_layout_03_amd as ep

    if op == "route":
        return ep.ep_route(s["logits"], c["K"], score=_score(ep, c), bias=s["bias"], num_groups=c["G"],
                           topk_groups=c["TG"], group_top=c["gtop"], renormalize=c["renorm"], scale=c["scale"],
                           token_mask=s["mask"])
    if op == "route_backward":
        return ep.ep_route_backward(s["gw"], s["logits"], s["idx"], score=_score(ep, c), renormalize=c["renorm"],
                                    scale=c["scale"])
    if op == "combine_backward":
        return ep.ep_combine_backward(s["go"], s["y"], s["layout"], s["w"], grad_y=s["gy"])
    tokens = c["rows"] == "tokens"
    if op == "lora":
        return ep.ep_lora(s["x"], s["layout"], s["a"], s["b"], base=s["base"], scales=s["scales"], gather=tokens,
                          scatter=tokens, out=s["out"])
    return ep.ep_lora_backward(s["go"], s["x"], s["layout"], s["a"], s["b"], scales=s["scales"], gather=tokens,
                               scatter=tokens, grad_x=s["gx"])


def _score(ep, c):
    return ep.EP_SCORE_SIGMOID if c["score"] == "sigmoid" else ep.EP_SCORE_SOFTMAX


# ------------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["T"]
    if op in ("route", "route_backward"):
        E, K = case["E"], case["K"]
        el = 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return {"bytes": T * E * el + T * K * 12, "flops": T * E * 4}
        return {"bytes": 2 * T * E * el + T * K * 12, "flops": T * E * 4}
    if op == "combine_backward":
        H, K = case["H"], case["K"]
        n = T * K * (1 - case["masked"])
        return {"bytes": T * H * 2 + 2 * n * H * 2 + T * K * 12, "flops": 3 * n * H}
    E, K, H, N, R = (case[k] for k in "EKHNR")
    n = T * K * (1 - case["none"])
    used = min(E, case["requests"] or T * K)
    if op == "lora":
        out_rows = T if case["rows"] == "tokens" else n
        return {"bytes": n * H * 2 + 2 * out_rows * N * 2 + used * R * (H + N) * 2 + n * 4,
                "flops": 2 * n * R * (H + N)}
    return {"bytes": 2 * n * H * 2 + n * N * 2 + used * R * (H + N) * 2 + E * R * (H + N) * 2 + n * 4,
            "flops": 6 * n * R * (H + N)}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward,
            "combine_backward": _exact_combine_backward, "lora": _exact_lora,
            "lora_backward": _exact_lora_backward}[case["op"]](s, case)


def _np64(t):
    return t.double().cpu().numpy()


def _sigmoid64(l):
    return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))


def _score64(l, kind):
    if kind == "sigmoid":
        return _sigmoid64(l)
    e = np.exp(l - l.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _exact_route(s, c):
    l = _np64(s["logits"])
    T, E = l.shape
    p = _score64(l, c["score"])
    pick = l.copy() if s["bias"] is None else p + _np64(s["bias"])
    pick[np.isneginf(l)] = -np.inf
    rows = np.arange(T)
    if c["G"]:
        n = E // c["G"]
        gv = pick if s["bias"] is not None or c["gtop"] == 1 else np.where(np.isneginf(l), -np.inf, p)
        total = np.full((T, c["G"]), -np.inf)
        for gi in range(c["G"]):
            part = np.sort(gv[:, gi * n:(gi + 1) * n], axis=1)[:, ::-1][:, : c["gtop"]]
            total[:, gi] = np.where(np.isneginf(part[:, 0]), -np.inf, np.where(np.isneginf(part), 0, part).sum(1))
        shut = np.ones((T, c["G"]), bool)
        left = total.copy()
        for _ in range(c["TG"]):
            best = left.argmax(1)  # the first of equal ones
            shut[rows, best] = False
            # a group that is taken must not be taken again
            left[rows, best] = np.nan
            left = np.where(np.isnan(left), -np.inf, left)
        pick[np.repeat(shut, n, axis=1)] = -np.inf
    idx = np.full((T, c["K"]), -1, np.int64)
    raw = np.zeros((T, c["K"]))
    for k in range(c["K"]):
        best = pick.argmax(1)
        ok = pick[rows, best] > -np.inf
        if s["mask"] is not None:
            ok &= s["mask"].cpu().numpy()
        idx[:, k] = np.where(ok, best, -1)
        raw[:, k] = np.where(ok, p[rows, best], 0.0)
        pick[rows, best] = -np.inf
    if c["renorm"]:
        raw = raw / np.maximum(raw.sum(1, keepdims=True), 1e-300)
    return torch.from_numpy(idx), torch.from_numpy(raw * c["scale"])


def _exact_route_backward(s, c):
    l, idx, g = _np64(s["logits"]), s["idx"].cpu().numpy(), _np64(s["gw"])
    T, E = l.shape
    p = _score64(l, c["score"])
    rows = np.arange(T)
    # d loss / d score, then through the scores
    chosen = np.stack([np.where(idx[:, k] >= 0, p[rows, idx[:, k]], 0.0) for k in range(c["K"])], 1)
    g = np.where(idx >= 0, g * c["scale"], 0.0)
    if c["renorm"]:
        total = np.maximum(chosen.sum(1, keepdims=True), 1e-300)
        g = np.where(idx >= 0, (g - (g * chosen).sum(1, keepdims=True) / total) / total, 0.0)
    dp = np.zeros((T, E))
    for k in range(c["K"]):
        ok = idx[:, k] >= 0
        dp[rows[ok], idx[ok, k]] += g[ok, k]
    if c["score"] == "sigmoid":
        d = dp * p * _sigmoid64(-l)
    else:
        d = p * (dp - (dp * p).sum(1, keepdims=True))
    return torch.from_numpy(d)


def _exact_combine_backward(s, c):
    T, K = c["T"], c["K"]
    gy = torch.zeros(T * K, c["H"], dtype=torch.float64, device=_dev())
    gw = torch.zeros(T, K, dtype=torch.float64, device=_dev())
    for k in range(K):
        for t0 in range(0, T, 2048):
            part = slice(t0, min(T, t0 + 2048))
            at = s["slot"][part, k]
            ok = at >= 0
            go = s["go"][part][ok].double()
            gy[at[ok]] = s["w"][part, k][ok].double()[:, None] * go
            got = torch.zeros(ok.numel(), dtype=torch.float64, device=_dev())
            got[ok] = (go * s["y"][at[ok]].double()).sum(1)
            gw[part, k] = got
    return gy, gw


def _each_adapter(s):
    """(expert, its rows of x, base and out) for every expert with rows."""
    r0 = 0
    for e, n in enumerate(s["seg"]["counts"].tolist()):
        if n:
            yield e, s["at"][r0:r0 + n]
        r0 += n


def _exact_lora(s, c):
    out = s["base"].double()
    if c["rows"] == "experts":
        out[s["seg"]["rows"]:] = 0.0
    for e, at in _each_adapter(s):
        low = s["x"][at].double() @ s["a"][e].double().T
        out[at] += s["scales"][e].double() * (low @ s["b"][e].double().T)
    return out


def _exact_lora_backward(s, c):
    gx = torch.zeros(s["gx"].shape, dtype=torch.float64, device=_dev())
    ga = torch.zeros(s["a"].shape, dtype=torch.float64, device=_dev())
    gb = torch.zeros(s["b"].shape, dtype=torch.float64, device=_dev())
    for e, at in _each_adapter(s):
        x, g = s["x"][at].double(), s["go"][at].double() * s["scales"][e].double()
        a, b = s["a"][e].double(), s["b"][e].double()
        gx[at] = (g @ b) @ a
        ga[e] = (g @ b).T @ x
        gb[e] = g.T @ (x @ a.T)
    return gx, ga, gb
