"""The operators around the FP8 GEMMs of a transformer layer: their cases, their plain forms and their definition in 64 bits.

  norm      residual addition, root-mean-square norm and 1x128 quantisation (the A operand of the next GEMM)
  norm_grad the norm's gradients
  append    rotation of queries and keys, and the append of keys and values to a paged cache held in 8 bits
  attention causal attention over that cache

Where `own` is false, run() computes an operator from elementary torch operations in 32 bits; where it is true, through
the package's entry points.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
BF16, FP32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ATTENTION_WORKSPACE_BYTES = (64 << 20) + (64 << 10)


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one user: launch latency. Hidden size 7168 is the K of this repository's dense shapes.
        {"name": "norm 1 row", "op": "norm", "rows": 1, "cols": 7168, "type": "bf16", "residual": True},
        # a training or prefill batch of 4096 tokens
        {"name": "norm 4096 rows", "op": "norm", "rows": 4096, "cols": 7168, "type": "bf16", "residual": True},
        # a ragged number of tokens, unrounded activations, the first norm of a network (nothing to add)
        {"name": "norm fp32", "op": "norm", "rows": 1537, "cols": 2048, "type": "fp32", "residual": False},
        # the backward of the 4096-token batch, with the gradient that arrives over the residual stream
        {"name": "norm grad 4096 rows", "op": "norm_grad", "rows": 4096, "cols": 7168, "type": "bf16", "residual": True},
        # a small ragged micro-batch in 32 bits
        {"name": "norm grad fp32", "op": "norm_grad", "rows": 333, "cols": 2048, "type": "fp32", "residual": False},
        # one decode step of 64 users
        {"name": "append decode", "op": "append", "batch": 64, "max_new": 1, "max_len": 4096, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "interleaved": False},
        # prompts of up to 2048 tokens that enter the cache together, in small pages
        {"name": "append prompts", "op": "append", "batch": 6, "max_new": 2048, "max_len": 2048, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "interleaved": True},
        # one user, a short conversation: latency
        {"name": "attend 1 user", "op": "attention", "batch": 1, "max_new": 1, "max_len": 777, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0},
        # a decode step of 64 users with conversations of all lengths
        {"name": "attend 64 users", "op": "attention", "batch": 64, "max_new": 1, "max_len": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0},
        # few users with very long documents, one key head for 8 query heads, and a few drafted tokens each to verify
        {"name": "attend long", "op": "attention", "batch": 2, "max_new": 4, "max_len": 131072, "heads": 16, "kv_heads": 2,
         "dim": 128, "page": 128, "window": 0},
        # a layer with a sliding window, small heads, every query head with a key head of its own
        {"name": "attend window", "op": "attention", "batch": 33, "max_new": 1, "max_len": 5000, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 32, "window": 1024},
        # a chunk of 2048 prompt tokens on top of what is cached
        {"name": "attend prompts", "op": "attention", "batch": 2, "max_new": 2048, "max_len": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        case = _draw(rng)
        wide = case["heads"] * case["dim"] if "heads" in case else 0
        side = (case["heads"] + 2 * case["kv_heads"]) * case["dim"] if wide else 0
        if 3072 not in (wide, side, *case.values()):  # no size here or in the queries and the projection's output is that one
            return case


def _draw(rng):
    op = rng.choice(["norm", "norm_grad", "append", "append", "attention", "attention", "attention"])
    if op in ("norm", "norm_grad"):
        cols = 128 * _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(8192, 4096 * 7168 // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "fp32"]) if rows * cols <= 1 << 24 else "bf16",
                "residual": rng.random() < 0.7}
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16] if kv_heads <= 4 else [1, 2, 3, 4])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128])}
    wide = heads * case["dim"]
    if op == "append":
        prompt = rng.random() < 0.5
        case["interleaved"] = rng.random() < 0.5
        case["batch"] = _log_int(rng, 1, 8 if prompt else 128)
        case["max_new"] = _log_int(rng, 2, min(2048, (8192 * 4096) // (wide * case["batch"]))) if prompt else 1
        case["max_len"] = case["max_new"] + _log_int(rng, 1, 4096)
        return case
    case["window"] = 0 if rng.random() < 0.7 else _log_int(rng, 16, 4096)
    kind = rng.choice(["decode", "decode", "draft", "prompt"])
    if kind == "prompt":
        case["batch"] = _log_int(rng, 1, 4)
        case["max_new"] = _log_int(rng, 17, 2048)
        room = (2 * 2048 * 8192 * 32 * 128) // (case["batch"] * case["max_new"] * wide)  # the listed chunk's work
        case["max_len"] = case["max_new"] + _log_int(rng, 1, max(1, min(8192, room - case["max_new"])))
    else:
        case["batch"] = _log_int(rng, 1, 128)
        case["max_new"] = 1 if kind == "decode" else rng.randint(2, 8)
        room = (64 * 8192 * 8 * 128) // (case["batch"] * kv_heads * case["dim"])  # the 64 users' cache
        case["max_len"] = case["max_new"] + _log_int(rng, 1, max(1, min(131072, room)))
    return case


def lengths(case):
    """(new tokens, cached and new tokens) of each sequence: part of the case, not of the seed. The first has the most."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, full = [], []
    for b in range(case["batch"]):
        n = case["max_new"] if b == 0 or case["max_new"] <= 8 else rng.randint(max(1, case["max_new"] // 4), case["max_new"])
        m = case["max_len"] if b == 0 else rng.randint(max(n, case["max_len"] // 16), case["max_len"])
        new.append(n)
        full.append(max(n, m))
    return new, full


# --------------------------------------------------------------------------------------------------------------- inputs

def _rotation(positions, half):
    """The rotation's table: cosines, then sines, of `half` frequencies at each position."""
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(FP32)


def _page_scale(amax):
    """The smallest power of two (2^-126 at least) by which `amax` fits e4m3, as a 32-bit float."""
    m, x = torch.frexp(amax)
    e = (x - 9 + (m > 0.875)).clamp(min=-126)
    e = torch.where(amax > 0, e, -126)
    return ((e.to(torch.int32) + 127) << 23).view(FP32)


def _cache(gen, pages, kv_heads, page, dim):
    """A cache as a server has it after a while: every page with its own scale, some channels larger than others."""
    spread = torch.rand(kv_heads, 1, dim, generator=gen, device="cuda") * 1.5 + 0.25
    codes = torch.empty(pages, kv_heads, page, dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, kv_heads, dtype=FP32, device="cuda")
    step = max(1, (1 << 26) // (kv_heads * page * dim))
    for i in range(0, pages, step):
        x = torch.randn(min(step, pages - i), kv_heads, page, dim, generator=gen, device="cuda") * spread
        s = _page_scale(x.abs().amax(dim=(2, 3)))
        codes[i:i + step] = (x / s[:, :, None, None]).to(FP8).view(torch.uint8)
        scales[i:i + step] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        dt = BF16 if case["type"] == "bf16" else FP32
        channel = torch.exp(randn(cols) * 0.5)
        st = {"op": op, "weight": (1.0 + 0.2 * randn(cols)).to(dt), "x": (randn(rows, cols) * channel).to(dt), "residual": None}
        if op == "norm":
            if case["residual"]:
                st["residual"] = (randn(rows, cols) * channel * 3).to(dt)
                st["h"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            st["q"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
            st["scale"] = torch.zeros(cols // 128, (rows + 3) // 4 * 4, dtype=FP32, device="cuda")
            st["rstd"] = torch.empty(rows, dtype=FP32, device="cuda")
        else:
            st["dy"] = (randn(rows, cols) * 0.01).to(dt)
            st["rstd"] = (st["x"].double().square().mean(dim=1) + EPS).rsqrt().to(FP32)
            if case["residual"]:
                st["residual"] = (randn(rows, cols) * 0.01).to(dt)
        return st

    B, Hq, Hkv, D, P = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    new, full = lengths(case)
    T, npages = sum(new), [-(-n // P) for n in full]
    pages = sum(npages) + sum(npages) // 8 + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, max(npages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(npages):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = {"op": op, "page": P, "max_new": max(new), "max_len": max(full), "table": table.cuda(),
          "seq_lens": torch.tensor(full, dtype=torch.int32, device="cuda"),
          "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"),
          "sequence": torch.repeat_interleave(torch.arange(B), torch.tensor(new)).cuda()}  # of each token
    st["k_cache"], st["k_scale"] = _cache(gen, pages, Hkv, P, D)
    st["v_cache"], st["v_scale"] = _cache(gen, pages, Hkv, P, D)
    if op == "append":  # the projection's output: queries, keys and values of a token side by side
        qkv = (randn(T, (Hq + 2 * Hkv) * D) * 1.5).to(BF16)
        st["qkv"] = qkv
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["rotation"] = _rotation(max(full), D // 2)
        st["interleaved"] = case["interleaved"]
        st["q_out"] = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
    else:
        st["q"] = (randn(T, Hq, D) * 2.5).to(BF16)
        st["out"] = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
        st["lse"] = torch.empty(T, Hq, dtype=FP32, device="cuda")
        st["softmax_scale"] = D ** -0.5
        st["window"] = case["window"]
        st["workspace"] = torch.zeros(ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------------------------------------------- plain forms

def _plain_norm(st):
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(h.dtype)
    x = h.float()
    rstd = 1.0 / (x.square().mean(dim=1) + EPS).sqrt()
    y = x * rstd[:, None] * st["weight"].float()
    y = y.view(x.shape[0], -1, 128)
    amax = y.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (y / scale[:, :, None]).to(FP8).view(x.shape)
    return {"q": q, "scale": scale.t(), "h": h if st["residual"] is not None else None, "rstd": rstd}


def _plain_norm_grad(st):
    xhat = st["x"].float() * st["rstd"][:, None]
    dy = st["dy"].float()
    g = dy * st["weight"].float()
    dx = st["rstd"][:, None] * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if st["residual"] is not None:
        dx = dx + st["residual"].float()
    return {"dx": dx.to(st["x"].dtype), "dw": (dy * xhat).sum(dim=0)}


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D]; cos, sin [T, 1, D / 2]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_store(cache, scales, x, st):
    """x [T, heads, D] into the pages that the new tokens fall in; a page whose new tokens need a larger scale than the
    earlier ones in it had is re-encoded."""
    P, start, cu = st["page"], st["seq_lens"].long() - st["cu_q"].diff().long(), st["cu_q"].long()
    last = (st["seq_lens"].long() - 1) // P
    n = (st["max_new"] + P - 2) // P + 1
    at = torch.minimum((start // P)[:, None] + torch.arange(n, device=x.device), last[:, None])  # a sequence with fewer repeats its last
    pages = st["table"].long().gather(1, at)
    slot = at[:, :, None] * P + torch.arange(P, device=x.device)
    is_new = (slot >= start[:, None, None]) & (slot < st["seq_lens"][:, None, None])
    is_old = slot < start[:, None, None]
    token = (cu[:-1, None, None] + slot - start[:, None, None]).clamp(0, x.shape[0] - 1)
    value = x[token].transpose(2, 3)  # [B, n, heads, P, D]
    is_new, is_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
    scale = _page_scale(torch.where(is_new, value.abs(), torch.zeros_like(value)).amax(dim=(3, 4)))
    before, bytes_before = scales[pages], cache[pages]
    scale = torch.where((at * P < start[:, None])[:, :, None], torch.maximum(scale, before), scale)
    s = scale[:, :, :, None, None]
    old = bytes_before.view(FP8).float() * (before[:, :, :, None, None] / s)
    code = torch.where(is_new, value / s, torch.where(is_old, old, torch.zeros_like(old))).to(FP8).view(torch.uint8)
    cache[pages] = torch.where(is_new | is_old, code, bytes_before)
    scales[pages] = scale


def _plain_append(st):
    position = (st["seq_lens"].long() - st["cu_q"][1:].long())[st["sequence"]] + torch.arange(st["sequence"].numel(), device="cuda")
    cos, sin = st["rotation"][position][:, None, :].chunk(2, dim=-1)
    q = _rotate(st["q"].float(), cos, sin, st["interleaved"]).to(BF16)
    k = _rotate(st["k"].float(), cos, sin, st["interleaved"])
    _plain_store(st["k_cache"], st["k_scale"], k, st)
    _plain_store(st["v_cache"], st["v_scale"], st["v"].float(), st)
    return q


def _plain_attention(st):
    (T, Hq, D), (B, n), P = st["q"].shape, st["table"].shape, st["page"]
    Hkv = st["k_cache"].shape[1]
    g, N, L = Hq // Hkv, st["max_new"], n * P
    pages = st["table"].long().clamp(min=0)

    def gathered(cache, scale):  # [B, n, Hkv, P, D]
        return cache.view(FP8)[pages].float() * scale[pages][:, :, :, None, None]

    length, cu = st["seq_lens"].long(), st["cu_q"].long()
    token = cu[:-1, None] + torch.arange(N, device="cuda")  # [B, N]
    position = length[:, None] - cu.diff()[:, None] + torch.arange(N, device="cuda")
    q = st["q"].float()[token.clamp(max=T - 1)].view(B, N, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B * Hkv, N * g, D)
    keys = gathered(st["k_cache"], st["k_scale"]).permute(0, 2, 4, 1, 3).reshape(B * Hkv, D, L)
    logits = torch.bmm(q, keys).mul_(st["softmax_scale"])
    key = torch.arange(L, device="cuda")
    seen = (key <= position[:, :, None]) & (key < length[:, None, None])
    if st["window"]:
        seen &= key > position[:, :, None] - st["window"]
    logits.view(B, Hkv, N, g, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = logits.amax(dim=2, keepdim=True).clamp(min=-1e30)
    weights = logits.sub_(top).exp_()
    total = weights.sum(dim=2, keepdim=True)
    values = gathered(st["v_cache"], st["v_scale"]).transpose(1, 2).reshape(B * Hkv, L, D)
    out = torch.bmm(weights, values) / total.clamp(min=1e-30)
    lse = (top + total.log()).view(B, Hkv, N, g).permute(0, 2, 1, 3).reshape(B, N, Hq)
    out = out.view(B, Hkv, N, g, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    index = torch.arange(T, device="cuda") - cu[st["sequence"]]
    return out[st["sequence"], index].to(BF16), lse[st["sequence"], index]


def run(state):
    st, op = state, state["op"]
    if own:
        import moe_grouped_gemm_fp32_amd as fg
    if op == "norm":
        if not own:
            return _plain_norm(st)
        fg.rmsnorm_quantize_1x128(st["x"], st["weight"], residual=st["residual"], eps=EPS, Q=st["q"], sa=st["scale"], H=st.get("h"),
                                  rstd=st["rstd"])
        return {"q": st["q"].view(FP8), "scale": st["scale"][:, :st["x"].shape[0]], "h": st.get("h"), "rstd": st["rstd"]}
    if op == "norm_grad":
        if not own:
            return _plain_norm_grad(st)
        dx, dw = fg.rmsnorm_backward(st["dy"], st["x"], st["rstd"], st["weight"], dH=st["residual"])
        return {"dx": dx, "dw": dw}
    if own:
        cache = fg.PagedKVCache(st["k_cache"], st["k_scale"], st["v_cache"], st["v_scale"])
    if op == "append":
        if own:
            q = fg.rope_append_paged_kv(st["q"], st["k"], st["v"], st["rotation"], cache, st["table"], st["seq_lens"], st["cu_q"],
                                        interleaved=st["interleaved"], q_out=st["q_out"])
        else:
            q = _plain_append(st)
        return {"q": q, "k_cache": st["k_cache"].view(FP8), "k_scale": st["k_scale"], "v_cache": st["v_cache"].view(FP8),
                "v_scale": st["v_scale"]}
    if own:
        out = fg.paged_attention(st["q"], cache, st["table"], st["seq_lens"], st["cu_q"], out=st["out"], lse=st["lse"],
                                 softmax_scale=st["softmax_scale"], window=st["window"], workspace=st["workspace"])
        lse = st["lse"]
    else:
        out, lse = _plain_attention(st)
    return {"out": out, "lse": lse}


# ----------------------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size = case["rows"] * case["cols"], 2 if case["type"] == "bf16" else 4
        if op == "norm":
            return {"bytes": n * (size * (3 if case["residual"] else 1) + 1) + n // 128 * 4 + case["rows"] * 4 + case["cols"] * size,
                    "flops": n * 9}
        return {"bytes": n * size * (4 if case["residual"] else 3) + case["rows"] * 4 + case["cols"] * (size + 4), "flops": n * 11}
    new, full = lengths(case)
    Hq, Hkv, D, P, T = case["heads"], case["kv_heads"], case["dim"], case["page"], sum(new)
    if op == "append":  # the new tokens' codes are written; the pages that were begun earlier have a scale to compare
        touched = sum(-(-m // P) - (m - n) // P for n, m in zip(new, full))
        return {"bytes": T * D * (2 * Hq * 2 + 2 * Hkv * 3) + T * D * 4 + touched * Hkv * 2 * 4, "flops": T * D * (3 * Hq + 8 * Hkv)}
    window = case["window"] or 1 << 60
    pairs = sum(sum(min(p + 1, window) for p in range(m - n, m)) for n, m in zip(new, full))
    read = sum(min(m, window + n - 1) for n, m in zip(new, full))  # keys that some token sees
    return {"bytes": 2 * read * Hkv * (D + 4 / P) + T * Hq * (D * 2 * 2 + 4), "flops": pairs * Hq * D * 4}


# ---------------------------------------------------------------------------------------------- the definition, 64 bits

def _exact_store(codes, scales, x, st):
    """Page by page: what each code stands for over its page's scale, before its rounding to 8 bits."""
    P = st["page"]
    value, scale = codes.view(FP8).double(), scales.double()
    new, full, table = st["cu_q"].diff().tolist(), st["seq_lens"].tolist(), st["table"].tolist()
    done = 0
    for b, (n, m) in enumerate(zip(new, full)):
        at = m - n
        while at < m:
            page, first = table[b][at // P], at % P
            count = min(P - first, m - at)
            rows = x[done:done + count].transpose(0, 1)  # [heads, count, D]
            fits = torch.tensor(2.0, dtype=torch.float64, device="cuda") ** torch.ceil(torch.log2(rows.abs().amax(dim=(1, 2)) / E4M3_MAX))
            fits = fits.clamp(min=2.0 ** -126)
            if first:
                fits = torch.maximum(fits, scale[page])
                value[page, :, :first] *= (scale[page] / fits)[:, None, None]
            scale[page] = fits
            value[page, :, first:first + count] = rows / fits[:, None, None]
            at, done = at + count, done + count
    return value, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = (h + st["residual"].double()).to(st["x"].dtype)  # the sum is stored, and normalised as stored
        x = h.double()
        rstd = (x.pow(2).sum(1) / x.shape[1] + EPS) ** -0.5
        blocks = (x * rstd[:, None] * st["weight"].double()).unflatten(1, (-1, 128))
        scale = blocks.abs().max(2).values / E4M3_MAX
        scale[scale == 0] = 1.0
        return {"q": (blocks / scale[..., None]).flatten(1), "scale": scale.t(), "h": h.double() if st["residual"] is not None else None,
                "rstd": rstd}
    if op == "norm_grad":
        r, w, x, dy = (st[k].double() for k in ("rstd", "weight", "x", "dy"))
        wdy = w * dy
        dx = r[:, None] * wdy - x * (r ** 3 / x.shape[1] * (wdy * x).sum(1))[:, None]
        if st["residual"] is not None:
            dx += st["residual"].double()
        return {"dx": dx, "dw": (dy * x).t() @ r}
    new, full = st["cu_q"].diff().tolist(), st["seq_lens"].tolist()
    if op == "append":
        half = st["rotation"].shape[1] // 2
        position = torch.cat([torch.arange(m - n, m) for n, m in zip(new, full)]).cuda()
        turn = st["rotation"].double()[position]
        turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]

        def rotated(x):
            x = x.double()
            pairs = x.unflatten(-1, (half, 2)) if st["interleaved"] else torch.stack([x[..., :half], x[..., half:]], -1)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            return y.flatten(-2) if st["interleaved"] else torch.cat([y[..., 0], y[..., 1]], -1)

        k_value, k_scale = _exact_store(st["k_cache"], st["k_scale"], rotated(st["k"]), st)
        v_value, v_scale = _exact_store(st["v_cache"], st["v_scale"], st["v"].double(), st)
        return {"q": rotated(st["q"]), "k_cache": k_value, "k_scale": k_scale, "v_cache": v_value, "v_scale": v_scale}
    T, Hq, D = st["q"].shape
    Hkv, P = st["k_cache"].shape[1], st["page"]
    g = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(new, full)):
        pages = st["table"][b, :-(-m // P)].long()
        key, position = torch.arange(m, device="cuda"), torch.arange(m - n, m, device="cuda")
        hidden = key[None] > position[:, None]
        if st["window"]:
            hidden |= key[None] <= position[:, None] - st["window"]
        for h in range(Hkv):
            k, v = ((c[pages, h].view(FP8).double() * s[pages, h].double()[:, None, None]).flatten(0, 1)[:m]
                    for c, s in ((st["k_cache"], st["k_scale"]), (st["v_cache"], st["v_scale"])))
            for i in range(h * g, h * g + g):
                logits = (st["q"][at:at + n, i].double() @ k.t() * st["softmax_scale"]).masked_fill(hidden, -math.inf)
                lse[at:at + n, i] = torch.logsumexp(logits, 1)
                out[at:at + n, i] = torch.softmax(logits, 1) @ v
        at += n
    return {"out": out, "lse": lse}
