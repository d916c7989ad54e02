"""Workloads of the attention-side operators: rotary positions with several axes
(forward, gradient, and fused with the write of K and V into a paged cache) and
attention over that cache (single tokens, chunks of new tokens, a sliding window
with sink tokens).

Each case is a plain dict. ``prepare`` builds the inputs on the GPU, ``run``
makes one pass: with ``own`` through the library's kernels, otherwise in plain
32-bit torch operations; ``exact`` gives the same outputs from the definition in
64 bits. Sizes: 32 heads of 128 are the 4096 columns of the benchmark's
projections, 64 heads of 128 its 8192 columns with 16 rows; the rest is generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------- the cases
def _rope(name, tokens, heads, dim, pairs, axes, interleaved, dtype):
    return {"name": name, "op": "rope_gradient", "tokens": tokens, "heads": heads, "dim": dim, "pairs": pairs,
            "axes": axes, "interleaved": interleaved, "type": dtype}


def _append(name, tokens, heads, kv_heads, dim, pairs, axes, interleaved, page, first, dtype):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "pairs": pairs, "axes": axes, "interleaved": interleaved, "page": page, "first": first, "type": dtype}


def _attention(name, batch, decoding, new, ctx, heads, kv_heads, dim, page, window, sinks, heads_first, dtype):
    return {"name": name, "op": "attention", "batch": batch, "decoding": decoding, "new": new, "ctx": ctx,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "sinks": sinks,
            "heads_first": heads_first, "type": dtype}


def listed():
    return [
        # one generated token of one sequence, straight from the 4096-column projections: latency only
        _append("append_token", 1, 32, 32, 128, 64, 1, False, 16, 1036, "f16"),
        # one token of each of 61 sequences, three position axes, shared K/V heads
        _append("append_batch", 61, 32, 8, 128, 64, 3, False, 16, 60000, "bf16"),
        # a long prompt of text and images: the bandwidth of the fused rotation and cache write
        _append("append_prompt", 8192, 32, 8, 128, 64, 3, False, 64, 0, "f16"),
        # training: the gradient through the rotation of 4099 tokens, adjacent pairs, 24 of 128 columns unrotated
        _rope("rope_gradient", 4099, 32, 128, 52, 3, True, "f16"),
        # one token of one sequence over a short, odd context, one K/V head for each query head: latency only
        _attention("decode_token", 1, 1, 1, 1037, 32, 32, 128, 16, 0, 0, False, "f16"),
        # a serving step: 64 sequences of unlike lengths, 4 query heads to a K/V head
        _attention("decode_batch", 64, 64, 1, 8192, 32, 8, 128, 16, 0, 0, False, "f16"),
        # one token over a very long context: the long axis has to be split over the whole GPU
        _attention("decode_long", 1, 1, 1, 131071, 32, 8, 128, 64, 0, 0, True, "bf16"),
        # 16 long sequences of 64 query heads that see a window of 4096 and 4 first tokens
        _attention("decode_window", 16, 16, 1, 32768, 64, 8, 128, 32, 4096, 4, False, "bf16"),
        # a short prompt's second piece: odd sizes, 5 query heads to a K/V head of 64 columns
        _attention("chunk_odd", 3, 0, 77, 613, 15, 3, 64, 16, 0, 0, False, "f16"),
        # a mixed serving step: 31 single tokens beside one chunk of 512 new tokens
        _attention("step_mixed", 32, 31, 512, 6000, 32, 8, 128, 16, 0, 0, False, "f16"),
        # 4096 new tokens on top of 12288: the arithmetic of a long prompt
        _attention("chunk_long", 1, 0, 4096, 16384, 32, 8, 128, 64, 0, 0, False, "f16"),
        # whole prompts of up to 4096 tokens with a window of 1024 and 4 first tokens
        _attention("prompt_window", 4, 0, 4096, 4096, 32, 8, 128, 32, 1024, 4, True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "rope_gradient", "decode", "decode", "chunk", "chunk", "mixed"])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128, 128, rng.choice([72, 80, 96, 112])])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind in ("append", "rope_gradient"):
        tokens = _log(rng, 1, 8192)
        pairs = rng.choice([dim // 2, dim // 2, dim // 4 + 1])
        axes, inter = rng.choice([1, 2, 3]), rng.random() < 0.5
        if kind == "append":
            return _append("", tokens, min(heads, 32), kv_heads, dim, pairs, axes, inter, page,
                           rng.randrange(100000), dtype) | {"name": "append"}
        return _rope("rope", tokens, min(heads, 32), dim, pairs, axes, inter, dtype)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    sinks = rng.choice([0, 4, 37]) if window else 0
    heads_first = rng.random() < 0.5
    if kind == "decode":
        ctx = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(128, (1 << 22) // (ctx * kv_heads))))
        return _attention("decode", batch, batch, 1, ctx, heads, kv_heads, dim, page, window, sinks, heads_first, dtype)
    new = _log(rng, 2, 3000)
    ctx = max(new, _log(rng, 2, 16000))
    batch = max(1, min(_log(rng, 1, 32), int(4.0e8 / (new * ctx * heads)), int(1.5e6 / (ctx * kv_heads))))
    decoding = batch - 1 if kind == "mixed" else 0
    return _attention(kind, batch, decoding, new, ctx, heads, kv_heads, dim, page, window, sinks, heads_first, dtype)


def _lengths(case):
    """(new tokens, positions in the cache) of each sequence; the first `decoding` ones have one new token."""
    b = case["batch"]
    new, kv = [], []
    for i in range(b):
        share = 1.0 - 0.75 * ((i * 7919) % b) / b
        n = 1 if i < case["decoding"] else max(1, int(case["new"] * (1.0 - 0.4 * ((b - 1 - i) % b) / b)))
        new.append(n)
        kv.append(max(n, int(case["ctx"] * share)))
    return new, kv


# ----------------------------------------------------------------- the inputs
def _sections(case):
    r, a = case["pairs"], case["axes"]
    parts = [r // a] * a
    parts[0] += r - sum(parts)
    return tuple(parts)


def _positions(case, first, gen):
    """int32 [axes, tokens]: text runs on along every axis; spans of image patches share a time and
    count rows and columns from where the text stopped."""
    t = case["tokens"]
    at = torch.arange(t, device="cuda", dtype=torch.int64)
    axes = [first + at]
    if case["axes"] > 1:
        width = 24
        start = first + (at // 480) * 480
        patch = (at // 480) % 2 == 1
        within = at % 480
        axes = [torch.where(patch, start, first + at)]
        axes.append(torch.where(patch, start + within // width, first + at))
        if case["axes"] > 2:
            axes.append(torch.where(patch, start + within % width, first + at))
    shift = torch.randint(0, 7, (1,), device="cuda", generator=gen)
    return (torch.stack(axes) + shift).to(torch.int32).contiguous()


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = TYPES[case["type"]]
    d = case["dim"]
    s = {"case": case}
    if case["op"] != "attention":
        t, r = case["tokens"], case["pairs"]
        s["sections"] = _sections(case)
        s["inv_freq"] = (10000.0 ** (-torch.arange(r, dtype=torch.float64) / r)).to(torch.float32).cuda()
        s["positions"] = _positions(case, case.get("first", 0), gen)
        if case["op"] == "rope_gradient":
            s["dy"] = _normal(gen, (t, case["heads"], d), dtype, 0.1)
            return s
        s["q"] = _normal(gen, (t, case["heads"], d), dtype)
        s["k"] = _normal(gen, (t, case["kv_heads"], d), dtype)
        s["v"] = _normal(gen, (t, case["kv_heads"], d), dtype)
        pages = -(-t // case["page"]) + 3
        shape = (pages, case["page"], case["kv_heads"], d)
        s["k_cache"], s["v_cache"] = _normal(gen, shape, dtype), _normal(gen, shape, dtype)
        # whole runs of slots in pages of a random order, as an allocator gives them
        order = torch.randperm(pages, device="cuda", generator=gen)
        at = torch.arange(t, device="cuda")
        s["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).to(torch.int32)
        return s
    new, kv = _lengths(case)
    page, hk = case["page"], case["kv_heads"]
    per = [-(-n // page) for n in kv]
    used = sum(per)
    pages = used + 2
    shape = (pages, hk, page, d) if case["heads_first"] else (pages, page, hk, d)
    kc, vc = _normal(gen, shape, dtype), _normal(gen, shape, dtype)
    if case["heads_first"]:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    s["k_cache"], s["v_cache"] = kc, vc
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.zeros((case["batch"], max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    s["page_table"] = table
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["q_starts"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    s["max_new"] = max(new)
    # queries of several lengths: softmaxes from nearly flat to sharply peaked
    q = torch.randn((sum(new), case["heads"], d), device="cuda", generator=gen)
    q *= torch.linspace(0.5, 3.0, case["heads"], device="cuda")[None, :, None]
    s["q"] = q.to(dtype)
    s["scale"] = 1.0 / math.sqrt(d)
    if own:
        from qkv_projection_gb300 import kaio
        s["workspace"] = kaio.paged_attention_workspace()
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _plain_attention(state) if op == "attention" else _plain_rope(state)


def _run_own(s):
    from qkv_projection_gb300 import kaio
    c = s["case"]
    if c["op"] == "rope_gradient":
        return {"dx": kaio.rope(s["dy"], s["positions"], s["inv_freq"], sections=s["sections"],
                                interleaved=c["interleaved"], inverse=True)}
    if c["op"] == "append":
        q = kaio.rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"],
                             s["slots"], sections=s["sections"], interleaved=c["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = kaio.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_starts"],
                                    max_new=s["max_new"], scale=s["scale"], window=c["window"], sinks=c["sinks"],
                                    workspace=s["workspace"], return_lse=True)
    return {"out": out, "lse": lse}


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] rotated in 32 bits; cos, sin [T, pairs]."""
    x = x.float()
    r = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * r:]), -1)


def _plain_rope(s):
    c = s["case"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=c["pairs"])
    angle = s["positions"].float()[axis].T * s["inv_freq"]
    cos, sin = torch.cos(angle), torch.sin(angle)
    if c["op"] == "rope_gradient":
        return {"dx": _rotate(s["dy"], cos, -sin, c["interleaved"]).to(s["dy"].dtype)}
    dtype = s["q"].dtype
    slots = s["slots"].long()
    at = (slots // c["page"], slots % c["page"])
    s["k_cache"][at] = _rotate(s["k"], cos, sin, c["interleaved"]).to(dtype)
    s["v_cache"][at] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, c["interleaved"]).to(dtype), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    b, hk, d, n = c["batch"], c["kv_heads"], c["dim"], s["max_new"]
    group = c["heads"] // hk
    kv = s["kv_lens"].long()
    starts = s["q_starts"].long()
    new = starts[1:] - starts[:-1]
    width = s["page_table"].shape[1] * c["page"]
    table = s["page_table"].long()
    k = s["k_cache"][table].reshape(b, width, hk, d).permute(0, 2, 3, 1).float()      # [b, hk, d, width]
    v = s["v_cache"][table].reshape(b, width, hk, d).permute(0, 2, 1, 3).float()      # [b, hk, width, d]
    i = torch.arange(n, device="cuda")
    real = i[None, :] < new[:, None]                                                  # [b, n]
    token = torch.where(real, starts[:-1, None] + i[None, :], 0)
    q = s["q"][token].float().reshape(b, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * n, d)
    pos = (kv - new)[:, None] + i[None, :]                                            # [b, n]
    j = torch.arange(width, device="cuda")
    seen = (j < kv[:, None, None]) & (j <= pos[:, :, None])
    if c["window"]:
        seen &= (j > pos[:, :, None] - c["window"]) | (j < c["sinks"])
    score = torch.matmul(q, k).reshape(b, hk, group, n, width)
    score *= s["scale"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0.0)
    out = torch.matmul(score.reshape(b, hk, group * n, width), v).reshape(b, hk, group, n, d)
    out /= torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, hk * group, d)[real].to(s["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(b, n, hk * group)[real]}


# ----------------------------------------------------------------- what a pass cannot do without
def _seen(n, kv, window, sinks):
    """(query-key pairs, distinct keys) that a sequence's n new tokens see."""
    p = np.arange(kv - n, kv, dtype=np.int64)
    if not window:
        return int((p + 1).sum()), kv
    lo = np.maximum(0, p - window + 1)
    first = np.minimum(sinks, lo)
    pairs = int((p + 1 - lo + first).sum())
    lo0 = max(0, kv - n - window + 1)
    return pairs, kv - lo0 + min(sinks, lo0)


def work(case):
    d = case["dim"]
    if case["op"] == "rope_gradient":
        values = case["tokens"] * case["heads"] * d
        return {"bytes": 4 * values + 4 * case["axes"] * case["tokens"] + 4 * case["pairs"],
                "flops": 6 * case["tokens"] * case["heads"] * case["pairs"]}
    if case["op"] == "append":
        t = case["tokens"]
        values = t * (case["heads"] + 2 * case["kv_heads"]) * d
        return {"bytes": 4 * values + 4 * (case["axes"] + 1) * t + 4 * case["pairs"],
                "flops": 6 * t * (case["heads"] + case["kv_heads"]) * case["pairs"]}
    new, kv = _lengths(case)
    seen = [_seen(n, k, case["window"], case["sinks"]) for n, k in zip(new, kv)]
    keys, pairs, tokens = sum(x[1] for x in seen), sum(x[0] for x in seen), sum(new)
    return {"bytes": 4 * tokens * case["heads"] * d + 4 * keys * case["kv_heads"] * d + 4 * tokens * case["heads"]
            + 4 * sum(-(-k // case["page"]) for k in kv) + 8 * case["batch"],
            "flops": 4 * d * case["heads"] * pairs}


# ----------------------------------------------------------------- the definition, in 64 bits
def _turn64(x, s):
    c = s["case"]
    sign = -1.0 if c["op"] == "rope_gradient" else 1.0
    y = x.double()
    out = y.clone()
    inv = s["inv_freq"].double().tolist()
    pair = 0
    for axis, count in enumerate(s["sections"]):
        at = s["positions"][axis].double()
        for _ in range(count):
            angle = at * inv[pair]
            co, si = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
            a, b = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + c["pairs"])
            out[..., a] = y[..., a] * co - y[..., b] * si
            out[..., b] = y[..., b] * co + y[..., a] * si
            pair += 1
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_gradient":
        return {"dx": _turn64(s["dy"], s)}
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        flat = s["slots"].long()
        kc.view(-1, *kc.shape[2:]).index_copy_(0, flat, _turn64(s["k"], s))
        vc.view(-1, *vc.shape[2:]).index_copy_(0, flat, s["v"].double())
        return {"q": _turn64(s["q"], s), "k_cache": kc, "v_cache": vc}
    new, kv = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        count = -(-length // case["page"])
        ids = s["page_table"][b, :count].long()
        keys = s["k_cache"][ids].flatten(0, 1)[:length]
        values = s["v_cache"][ids].flatten(0, 1)[:length]
        j = torch.arange(length, device="cuda")
        step = max(1, (1 << 27) // (length * group))
        for h in range(case["kv_heads"]):
            kh, vh = keys[:, h].double(), values[:, h].double()
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                p = torch.arange(length - n + i0, length - n + i1, device="cuda")[:, None]
                hidden = j > p
                if case["window"]:
                    hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
                rows, heads = slice(row + i0, row + i1), slice(h * group, (h + 1) * group)
                x = torch.einsum("igd,jd->igj", s["q"][rows, heads].double(), kh) * s["scale"]
                x = x.masked_fill(hidden[:, None, :], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[rows, heads] = z
                out[rows, heads] = torch.einsum("igj,jd->igd", torch.exp(x - z[..., None]), vh)
        row += n
    return {"out": out, "lse": lse}
