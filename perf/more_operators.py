"""The operators of a mixture-of-experts decoder layer around its GEMMs, attention and cache: their cases, their plain
forms and their definition in 64 bits.

  route     scores of experts, the choice among them and the weights of the chosen; the gradient of the logits
  dispatch  tokens' 8-bit rows laid out by expert, as the grouped GEMMs read them; the same rows gathered again, weighted
  combine   the experts' rows weighted and summed back to tokens; its gradients
  heads     norm of queries and keys for each head and their rotation in one pass; its gradients

Where `own` is false, run() computes an operator from elementary torch operations in 32 bits (the choice of experts in
64); where it is true, through the package's entry points.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
BF16, FP32, FP64, FP8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.int32
TYPE = {"bf16": BF16, "fp32": FP32}


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one user: latency. 256 experts and 8 of them a token are this repository's MoE workload.
        {"name": "route 1 token", "op": "route", "grad": False, "tokens": 1, "experts": 256, "top_k": 8, "scoring": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "offline": 0, "type": "fp32", "renormalize": True},
        # a training batch's tokens, balanced by a bias, in groups of experts
        {"name": "route 16384 tokens", "op": "route", "grad": False, "tokens": 16384, "experts": 256, "top_k": 8,
         "scoring": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "offline": 0, "type": "fp32",
         "renormalize": True},
        # the backward pass of a softmax router with a loss on its scores; a ragged batch, a number of experts that is no power of 2
        {"name": "route grad", "op": "route", "grad": True, "tokens": 10007, "experts": 160, "top_k": 6, "scoring": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "offline": 0, "type": "bf16", "renormalize": True},
        # a decode step of 64 users into the layout of the masked GEMM
        {"name": "dispatch decode", "op": "dispatch", "again": False, "tokens": 64, "experts": 256, "top_k": 8, "cols": 7168, "max_m": 64},
        # 4096 tokens of a prefill or training batch into the contiguous layout
        {"name": "dispatch 4096 tokens", "op": "dispatch", "again": False, "tokens": 4096, "experts": 256, "top_k": 8, "cols": 7168,
         "max_m": 0},
        # the rows of a gradient, weighted, into a layout that is there; ragged, few experts
        {"name": "gather gradient", "op": "dispatch", "again": True, "tokens": 1999, "experts": 24, "top_k": 6, "cols": 2048, "max_m": 0},
        # a decode step of 64 users out of the layout of the masked GEMM
        {"name": "combine decode", "op": "combine", "grad": False, "tokens": 64, "experts": 256, "top_k": 8, "cols": 7168, "max_m": 64,
         "addend": False, "type": "bf16"},
        # 4096 tokens, added to the residual stream
        {"name": "combine 4096 tokens", "op": "combine", "grad": False, "tokens": 4096, "experts": 256, "top_k": 8, "cols": 7168,
         "max_m": 0, "addend": True, "type": "bf16"},
        # the backward pass of the 4096 tokens
        {"name": "combine grad", "op": "combine", "grad": True, "tokens": 4096, "experts": 256, "top_k": 8, "cols": 7168, "max_m": 0,
         "addend": False, "type": "bf16"},
        # one decode step of 64 users
        {"name": "heads decode", "op": "heads", "grad": False, "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128, "rotated": 128,
         "interleaved": False, "type": "bf16"},
        # 8192 prompt tokens, half of every head rotated
        {"name": "heads 8192 tokens", "op": "heads", "grad": False, "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotated": 64, "interleaved": True, "type": "bf16"},
        # the backward pass of a ragged batch, every query head with a key head of its own
        {"name": "heads grad", "op": "heads", "grad": True, "tokens": 5003, "heads": 16, "kv_heads": 16, "dim": 64, "rotated": 64,
         "interleaved": False, "type": "bf16"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "combine", "heads"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        experts = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        offline = rng.choice([0, 0, rng.randint(1, max(1, experts // 8))])
        room = top_groups * (experts // groups) - offline  # experts that the worst choice of groups leaves
        return {"op": op, "grad": rng.random() < 0.35, "tokens": _log_int(rng, 1, min(32768, 16384 * 256 // experts)), "experts": experts,
                "top_k": rng.randint(1, max(1, min(16, room))), "scoring": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_best": rng.choice([1, 2]),
                "offline": offline if room > 0 else 0, "type": rng.choice(["fp32", "bf16"]), "renormalize": rng.random() < 0.7}
    if op == "heads":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        room = 8192 * 40 * 128 // ((heads + kv_heads) * dim)
        grad = rng.random() < 0.4
        kind = rng.choice(["bf16", "bf16", "fp32"])
        room //= (2 if grad else 1) * (2 if kind == "fp32" else 1)
        return {"op": op, "grad": grad, "tokens": _log_int(rng, 1, min(16384, room)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotated": rng.choice([dim, dim, dim // 2, 16, 48]), "interleaved": rng.random() < 0.5, "type": kind}
    experts = _log_int(rng, 4, 256)
    top_k = rng.randint(1, min(10, experts))
    cols = 128 * _log_int(rng, 1, 56)
    kind = rng.choice(["bf16", "bf16", "fp32"]) if op == "combine" else ""
    grad = op == "combine" and rng.random() < 0.4
    room = 4096 * 8 * 7168 // (top_k * cols) // (2 if kind == "fp32" else 1)
    tokens = _log_int(rng, 1, min(8192, room))
    case = {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "cols": cols, "max_m": 0}
    if rng.random() < 0.4:  # room for every token at an expert, or too little at the popular ones
        case["max_m"] = min(tokens, 256) if rng.random() < 0.7 else max(1, tokens * top_k // experts)
    if op == "dispatch":
        case["again"] = rng.random() < 0.3
    else:
        case.update(grad=grad, addend=not grad and rng.random() < 0.5, type=kind)
    return case


def layout_rows(case):
    """Rows of the expanded layout: for the contiguous one the most that the experts' segments, each rounded up to 128 rows, can take."""
    n, E = case["tokens"] * case["top_k"], case["experts"]
    if case["max_m"]:
        return E * case["max_m"]
    return (n + min(n, E) * 127) // 128 * 128


# --------------------------------------------------------------------------------------------------------------- inputs

def _popular(gen, tokens, experts, top_k):
    """Chosen experts of each token, some far more popular than others; a token's are distinct."""
    rank = torch.randperm(experts, generator=gen, device="cuda") + 1
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    return (noise - 0.7 * torch.log(rank.float())).topk(top_k, dim=1).indices.to(I32)


def _placed(ids, experts, max_m, rows):
    """(positions, counts, starts) of the choices ids [T, k], in the order of tokens within an expert."""
    flat = ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(experts, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    first = counts.cumsum(0) - counts
    if max_m:
        starts = torch.arange(experts, device="cuda") * max_m
        most = max_m
    else:
        padded = (counts + 127) // 128 * 128
        starts = padded.cumsum(0) - padded
        most = rows
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device="cuda") - first[flat[order]]
    positions = torch.where(rank < most, starts[flat] + rank, -1)
    return positions.to(I32).view(ids.shape), counts.clamp(max=most).to(I32), starts


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, T = case["op"], case["tokens"]
    st = {"op": op, "case": case}
    if op == "route":
        E, k = case["experts"], case["top_k"]
        st["logits"] = (randn(T, E) * 1.5 + randn(E) * 0.5).to(TYPE[case["type"]])
        if case["offline"]:
            st["logits"][:, torch.randperm(E, generator=gen, device="cuda")[:case["offline"]]] = -math.inf
        st["bias"] = randn(E) * 0.05 if case["bias"] else None
        st["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
        if case["grad"]:
            live = (st["logits"].float() + 1.5 * randn(T, E)).topk(k, dim=1).indices  # near the best
            st["ids"] = live.to(I32)
            st["dweights"] = randn(T, k) * 0.02
            st["dscores"] = randn(T, E) * 0.001 if case["scoring"] == "softmax" else None
            st["dlogits"] = torch.empty_like(st["logits"])
        else:
            st["ids"] = torch.empty(T, k, dtype=I32, device="cuda")
            st["weights"] = torch.empty(T, k, dtype=FP32, device="cuda")
        return st

    if op == "heads":
        Hq, Hk, D, R, dt = case["heads"], case["kv_heads"], case["dim"], case["rotated"], TYPE[case["type"]]
        qkv = (randn(T, (Hq + 2 * Hk) * D) * torch.exp(randn((Hq + 2 * Hk) * D) * 0.3)).to(dt)  # the projection's output
        st["q"], st["k"] = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        st["qw"], st["kw"] = ((1.0 + 0.2 * randn(D)).to(dt) for _ in range(2))
        span = 4096
        freq = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=FP64) / (R // 2))
        angle = torch.arange(span, device="cuda", dtype=FP64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(FP32)
        st["positions"] = (torch.arange(T, device="cuda") + int(torch.randint(span, (1,), generator=gen, device="cuda")))
        st["positions"] = (st["positions"] % span).to(I32)
        if case["grad"]:
            st["dq"], st["dk"] = (randn(T, Hq, D) * 0.01).to(dt), (randn(T, Hk, D) * 0.01).to(dt)
        else:
            st["q_out"], st["k_out"] = (torch.empty(T, h, D, dtype=dt, device="cuda") for h in (Hq, Hk))
        return st

    E, k, cols, max_m = case["experts"], case["top_k"], case["cols"], case["max_m"]
    rows = layout_rows(case)
    ids = _popular(gen, T, E, k)
    weights = rand(T, k) + 0.05
    weights = weights / weights.sum(dim=1, keepdim=True) * 2.5
    if op == "dispatch":
        x = (randn(T, cols) * torch.exp(randn(cols) * 0.5)).view(T, -1, 128)
        scale = x.abs().amax(dim=2) / E4M3_MAX
        st["q"] = (x / scale[:, :, None]).to(FP8).view(torch.uint8).view(T, cols)
        st["sa"] = torch.zeros(cols // 128, (T + 3) // 4 * 4, dtype=FP32, device="cuda")
        st["sa"][:, :T] = scale.t()
        st["ids"], st["weights"] = ids, weights if case["again"] else None
        shape = (E, max_m) if max_m else (rows,)
        ld = ((max_m or rows) + 3) // 4 * 4
        st["qx"] = torch.zeros(*shape, cols, dtype=torch.uint8, device="cuda")
        st["sax"] = torch.zeros(*shape[:-1], cols // 128, ld, dtype=FP32, device="cuda")
        positions, counts, starts = _placed(ids, E, max_m, rows)
        sources = torch.full((rows,), -1, dtype=I32, device="cuda")
        there = positions.flatten() >= 0
        sources[positions.flatten()[there].long()] = torch.arange(T * k, dtype=I32, device="cuda")[there]
        expert = None
        if not max_m:
            expert = torch.full((rows,), -1, dtype=I32, device="cuda")
            expert[positions.flatten().long()] = ids.flatten()
        given = (positions, sources, expert, counts)
        # a layout that is there is read; one that the call makes is written
        st["layout"] = given if case["again"] else tuple(None if t is None else torch.empty_like(t) for t in given)
        return st
    dt = TYPE[case["type"]]
    st["positions"], _, _ = _placed(ids, E, max_m, rows)
    st["weights"] = weights
    st["y"] = randn(rows, cols).to(dt)
    if max_m:
        st["y"] = st["y"].view(E, max_m, cols)
    if case["grad"]:
        st["do"] = (randn(T, cols) * 0.02).to(dt)
        st["dy"] = torch.zeros_like(st["y"])
        st["dweights"] = torch.empty(T, k, dtype=FP32, device="cuda")
    else:
        st["c"] = randn(T, cols).to(dt) if case["addend"] else None
        st["out"] = torch.empty(T, cols, dtype=dt, device="cuda")
    return st


# --------------------------------------------------------------------------------------------------------- plain forms

def _scores(x, scoring):
    if scoring == "sigmoid":
        return 1.0 / (1.0 + (-x).exp())
    e = (x - x.amax(dim=1, keepdim=True)).exp()
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(st):
    c = st["case"]
    T, E, k, G = c["tokens"], c["experts"], c["top_k"], c["groups"]
    x = st["logits"].double()  # 64 bits: which of two near scores is larger
    s = _scores(x, c["scoring"])
    key = s if st["bias"] is None else s + st["bias"].double()
    key = torch.where(x == -math.inf, -math.inf, key)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_best"]]
        group = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(dim=2))
        kept = group.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    value, ids = key.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > -math.inf
    w = torch.where(there, s.gather(1, ids), 0.0)
    if c["renormalize"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    return {"ids": torch.where(there, ids, -1).to(I32), "weights": (w * st["scale"]).to(FP32)}


def _plain_route_grad(st):
    c = st["case"]
    s = _scores(st["logits"].float(), c["scoring"])
    ids, g = st["ids"].long(), st["dweights"]
    chosen = s.gather(1, ids)
    if c["renormalize"]:
        total = chosen.sum(dim=1, keepdim=True) + 1e-20
        g = (g - (g * chosen).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros_like(s) if st["dscores"] is None else st["dscores"].clone()
    ds.scatter_add_(1, ids, g * st["scale"])
    dx = ds * s * (1.0 - s) if c["scoring"] == "sigmoid" else s * (ds - (ds * s).sum(dim=1, keepdim=True))
    return {"dlogits": dx.to(st["logits"].dtype)}


def _plain_dispatch(st):
    c = st["case"]
    k, max_m = c["top_k"], c["max_m"]
    qx, sax = st["qx"], st["sax"]
    positions, sources, expert, counts = st["layout"]
    if not c["again"]:
        placed, n, _ = _placed(st["ids"], c["experts"], max_m, sources.numel())
        positions.copy_(placed)
        counts.copy_(n)
        sources.fill_(-1)
        if max_m:  # what does not fit is left out
            at = torch.where(placed < 0, sources.numel(), placed).flatten().long()
            sources.copy_(torch.cat([sources, sources[:1]]).scatter_(0, at, torch.arange(at.numel(), dtype=I32, device="cuda"))[:-1])
        else:
            sources[placed.flatten().long()] = torch.arange(placed.numel(), dtype=I32, device="cuda")
            expert.fill_(-1)
            expert[placed.flatten().long()] = st["ids"].flatten()
    live = (sources >= 0).nonzero().flatten()
    source = sources[live].long()
    token = source // k
    qx.view(-1, c["cols"])[live] = st["q"][token]
    scale = st["sa"][:, token]
    if st["weights"] is not None:
        scale = scale * st["weights"].flatten()[source]
    if max_m:
        sax[live // max_m, :, live % max_m] = scale.t()
    else:
        sax[:, live] = scale
    return st["layout"]


def _plain_combine(st):
    c = st["case"]
    y = st["y"].view(-1, c["cols"])
    at = st["positions"].long()
    out = torch.zeros(c["tokens"], c["cols"], dtype=FP32, device="cuda") if st["c"] is None else st["c"].float()
    for j in range(c["top_k"]):
        w = torch.where(at[:, j] >= 0, st["weights"][:, j], 0.0)
        out = out + w[:, None] * y[at[:, j].clamp(min=0)].float()
    return {"out": out.to(y.dtype)}


def _plain_combine_grad(st):
    c = st["case"]
    y, dy, do = st["y"].view(-1, c["cols"]), st["dy"].view(-1, c["cols"]), st["do"].float()
    at = st["positions"].long()
    dw = torch.empty(c["tokens"], c["top_k"], dtype=FP32, device="cuda")
    for j in range(c["top_k"]):
        there = at[:, j] >= 0
        dw[:, j] = torch.where(there, (do * y[at[:, j].clamp(min=0)].float()).sum(dim=1), 0.0)
        rows = (st["weights"][:, j, None] * do).to(y.dtype)
        if c["max_m"]:
            dy[at[:, j][there]] = rows[there]
        else:
            dy[at[:, j]] = rows
    return {"dy": st["dy"], "dweights": dw}


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D] with the first 2 n columns turned; cos, sin [T, 1, n]."""
    n = cos.shape[-1]
    turned, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :n], turned[..., n:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_heads(st):
    cos, sin = st["cos_sin"][st["positions"].long()][:, None, :].chunk(2, dim=-1)
    out = {}
    for name, w in (("q", "qw"), ("k", "kw")):
        x = st[name].float()
        n = x / (x.square().mean(dim=2, keepdim=True) + EPS).sqrt() * st[w].float()
        out[name] = _rotate(n, cos, sin, st["case"]["interleaved"]).to(st[name].dtype)
    return out


def _plain_heads_grad(st):
    cos, sin = st["cos_sin"][st["positions"].long()][:, None, :].chunk(2, dim=-1)
    out = {}
    for name, w in (("q", "qw"), ("k", "kw")):
        x = st[name].float()
        rstd = 1.0 / (x.square().mean(dim=2, keepdim=True) + EPS).sqrt()
        xhat = x * rstd
        dn = _rotate(st["d" + name].float(), cos, -sin, st["case"]["interleaved"])
        g = dn * st[w].float()
        out["d" + name] = (rstd * (g - xhat * (g * xhat).mean(dim=2, keepdim=True))).to(st[name].dtype)
        out["d" + w] = (dn * xhat).sum(dim=(0, 1))
    return out


def run(state):
    st, op = state, state["op"]
    c = st["case"]
    if own:
        import moe_grouped_gemm_fp32_amd as fg
    if op == "route":
        if c["grad"]:
            if not own:
                return _plain_route_grad(st)
            return {"dlogits": fg.moe_route_backward(st["dweights"], st["logits"], st["ids"], scoring=c["scoring"],
                                                     renormalize=c["renormalize"], scale=st["scale"], dscores=st["dscores"],
                                                     dlogits=st["dlogits"])}
        if not own:
            return _plain_route(st)
        ids, weights = fg.moe_route(st["logits"], c["top_k"], bias=st["bias"], scoring=c["scoring"], groups=c["groups"],
                                    top_groups=c["top_groups"], group_best=c["group_best"], renormalize=c["renormalize"],
                                    scale=st["scale"], ids=st["ids"], weights=st["weights"])
        return {"ids": ids, "weights": weights}
    if op == "dispatch":
        if own:
            layout = fg.MoeLayout(*st["layout"])
            if c["again"]:
                fg.moe_gather(st["q"], st["sa"], layout, weights=st["weights"], Qx=st["qx"], sax=st["sax"])
            else:
                fg.moe_dispatch(st["q"], st["sa"], st["ids"], c["experts"], max_m=c["max_m"] or None, Qx=st["qx"], sax=st["sax"],
                                layout=layout)
        else:
            layout = _plain_dispatch(st)
        positions, sources, expert, counts = layout
        return {"qx": st["qx"].view(FP8), "sax": st["sax"], "positions": positions, "sources": sources, "experts": expert, "counts": counts}
    if op == "combine":
        if c["grad"]:
            if not own:
                return _plain_combine_grad(st)
            dy, dw = fg.moe_combine_backward(st["do"], st["y"], st["positions"], st["weights"], dY=st["dy"], dweights=st["dweights"])
            return {"dy": dy, "dweights": dw}
        if not own:
            return _plain_combine(st)
        return {"out": fg.moe_combine(st["y"], st["positions"], st["weights"], C=st["c"], out=st["out"])}
    if c["grad"]:
        if not own:
            return _plain_heads_grad(st)
        dq, dk, dqw, dkw = fg.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["qw"], st["kw"], st["cos_sin"],
                                                    st["positions"], eps=EPS, interleaved=c["interleaved"])
        return {"dq": dq, "dqw": dqw, "dk": dk, "dkw": dkw}
    if not own:
        return _plain_heads(st)
    q, k = fg.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["cos_sin"], st["positions"], eps=EPS,
                           interleaved=c["interleaved"], q_out=st["q_out"], k_out=st["k_out"])
    return {"q": q, "k": k}


# ----------------------------------------------------------------------------------------------------------------- work

def work(case):
    op, T = case["op"], case["tokens"]
    if op == "route":
        E, k, size = case["experts"], case["top_k"], 2 if case["type"] == "bf16" else 4
        if case["grad"]:
            scores = T * E * 4 if case["scoring"] == "softmax" else 0
            return {"bytes": 2 * T * E * size + scores + T * k * 8, "flops": T * (E * 8 + k * 6)}
        return {"bytes": T * E * size + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": T * E * 5}
    if op == "heads":
        D, size = case["dim"], 2 if case["type"] == "bf16" else 4
        n = T * (case["heads"] + case["kv_heads"]) * D
        table = min(T, 4096) * case["rotated"] * 4 + T * 4
        if case["grad"]:
            return {"bytes": 3 * n * size + table + 2 * D * (size + 4), "flops": n * 16}
        return {"bytes": 2 * n * size + table + 2 * D * size, "flops": n * 8}
    E, k, cols, n = case["experts"], case["top_k"], case["cols"], case["tokens"] * case["top_k"]
    placed = n if not case["max_m"] else min(n, E * case["max_m"])
    if op == "dispatch":
        row = cols + cols // 128 * 4
        rows = layout_rows(case)
        lists = n * 4 + rows * 4 + (0 if case["max_m"] else rows * 4) + E * 4  # the layout
        return {"bytes": (T + placed) * row + lists + n * 4, "flops": placed * cols // 128 if case["again"] else 0}
    size = 2 if case["type"] == "bf16" else 4
    if case["grad"]:
        return {"bytes": (2 * placed + T) * cols * size + n * 12, "flops": placed * cols * 3}
    return {"bytes": (placed + T * (2 if case["addend"] else 1)) * cols * size + n * 8, "flops": placed * cols * 2}


# ---------------------------------------------------------------------------------------------- the definition, 64 bits

def _exact_scores(x, scoring):
    return torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["tokens"]
    if op == "route":
        x = st["logits"].double()
        s = _exact_scores(x, case["scoring"])
        if case["grad"]:
            s = s.detach().requires_grad_()
            ids = st["ids"].long()
            chosen = s.gather(1, ids)
            w = st["scale"] * (chosen / (chosen.sum(1, keepdim=True) + 1e-20) if case["renormalize"] else chosen)
            loss = (w * st["dweights"].double()).sum()
            if st["dscores"] is not None:
                loss = loss + (s * st["dscores"].double()).sum()
            ds, = torch.autograd.grad(loss, s)
            s = s.detach()
            return {"dlogits": ds * s - ds * s * s if case["scoring"] == "sigmoid" else s * ds - s * (s * ds).sum(1, keepdim=True)}
        E, G, size = case["experts"], case["groups"], case["experts"] // case["groups"]
        key = s.clone() if st["bias"] is None else s + st["bias"].double()
        key[torch.isneginf(x)] = -math.inf
        if G > 1:  # groups in the order of their scores, one after another
            score = torch.empty(T, G, dtype=FP64, device="cuda")
            for g in range(G):
                part = key[:, g * size:(g + 1) * size].clone()
                score[:, g] = part.amax(1)
                if case["group_best"] == 2 and size > 1:
                    part.scatter_(1, part.argmax(1, keepdim=True), -math.inf)
                    second = part.amax(1)
                    score[:, g] += torch.where(torch.isneginf(second), 0.0, second)
            dropped = torch.ones(T, G, dtype=torch.bool, device="cuda")
            for _ in range(case["top_groups"]):
                first = (score == score.amax(1, keepdim=True)).logical_and(dropped).to(torch.int8).argmax(1, keepdim=True)
                dropped.scatter_(1, first, False)
                score.scatter_(1, first, -math.inf)
            key.view(T, G, size).masked_fill_(dropped[:, :, None], -math.inf)
        ids, w = [], []
        for _ in range(case["top_k"]):
            top = key.amax(1, keepdim=True)
            first = (key == top).to(torch.int8).argmax(1, keepdim=True)
            none = torch.isneginf(top)
            ids.append(torch.where(none, -1, first))
            w.append(torch.where(none, 0.0, s.gather(1, first)))
            key.scatter_(1, first, -math.inf)
        ids, w = torch.cat(ids, 1), torch.cat(w, 1)
        if case["renormalize"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return {"ids": ids.to(I32), "weights": w * st["scale"]}
    if op == "heads":
        table = st["cos_sin"].double()[st["positions"].long()]
        n = case["rotated"] // 2
        turn = torch.complex(table[:, :n], table[:, n:])[:, None]

        def rotated(x, turn):
            head, rest = x[..., :2 * n], x[..., 2 * n:]
            pairs = head.unflatten(-1, (n, 2)) if case["interleaved"] else torch.stack([head[..., :n], head[..., n:]], -1)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            y = y.flatten(-2) if case["interleaved"] else torch.cat([y[..., 0], y[..., 1]], -1)
            return torch.cat([y, rest], -1)

        out = {}
        for name, w in (("q", "qw"), ("k", "kw")):
            x, weight = st[name].double(), st[w].double()
            rstd = (x.pow(2).sum(2, keepdim=True) / case["dim"] + EPS) ** -0.5
            if not case["grad"]:
                out[name] = rotated(x * rstd * weight, turn)
                continue
            dn = rotated(st["d" + name].double(), turn.conj())
            out["d" + name] = rstd * dn * weight - x * rstd ** 3 * ((dn * weight * x).sum(2, keepdim=True) / case["dim"])
            out["d" + w] = (dn * x * rstd).flatten(0, 1).sum(0)
        return out
    k, cols = case["top_k"], case["cols"]
    if op == "dispatch":  # expert by expert
        positions, sources, expert, counts = (None if t is None else t.clone() for t in st["layout"])
        rows = sources.numel()
        token_of = torch.arange(T * k, device="cuda") // k
        value, scale = torch.zeros(rows, cols, dtype=FP32, device="cuda"), st["sax"].double()
        code, flat, at = st["q"].view(FP8).float(), st["ids"].flatten(), 0
        positions.fill_(-1)
        sources.fill_(-1)
        if expert is not None:
            expert.fill_(-1)
        for e in range(case["experts"]):
            choice = (flat == e).nonzero().flatten()
            if case["max_m"]:
                at, choice = e * case["max_m"], choice[:case["max_m"]]
            m = choice.numel()
            positions.view(-1)[choice] = torch.arange(at, at + m, dtype=I32, device="cuda")
            sources[at:at + m] = choice.to(I32)
            counts[e] = m
            value[at:at + m] = code[token_of[choice]]
            part = st["sa"].double()[:, token_of[choice]]
            if st["weights"] is not None:
                part = part * st["weights"].double().flatten()[choice]
            if case["max_m"]:
                scale[e, :, :m] = part
            else:
                scale[:, at:at + m] = part
                expert[at:at + m] = e
                at += -(-m // 128) * 128
        return {"qx": value.view(st["qx"].shape).to(FP64) if rows * cols <= 1 << 28 else value.view(st["qx"].shape), "sax": scale,
                "positions": positions, "sources": sources, "experts": expert, "counts": counts}
    y, at, w = st["y"].view(-1, cols), st["positions"].long(), st["weights"].double()
    if case["grad"]:
        dy, dw = torch.zeros(y.shape, dtype=FP64, device="cuda"), torch.zeros(T, k, dtype=FP64, device="cuda")
        for t in range(0, T, 512):  # some tokens at a time
            do, p = st["do"][t:t + 512].double(), at[t:t + 512]
            there = p >= 0
            dw[t:t + 512] = (y[p.clamp(min=0)].double() @ do[:, :, None])[:, :, 0].masked_fill(~there, 0.0)
            dy[p[there]] = (w[t:t + 512, :, None] * do[:, None])[there]
        return {"dy": dy.view(st["y"].shape), "dweights": dw}
    out = torch.zeros(T, cols, dtype=FP64, device="cuda") if st["c"] is None else st["c"].double()
    for t in range(0, T, 512):
        p = at[t:t + 512]
        weight = w[t:t + 512].masked_fill(p < 0, 0.0)
        out[t:t + 512] += (weight[:, None] @ y[p.clamp(min=0)].double())[:, 0]
    return {"out": out}
