"""Workloads of the paged cache's upkeep (copying, forking, appending, truncating and
compacting its pages) and of attention over it with capped scores, a bias that grows
with distance, and document and prefix masks.

Each case is a plain dict. ``prepare`` builds the inputs on the GPU, ``run`` makes one
pass: with ``own`` through the library's kernels, otherwise in plain torch operations
(32-bit arithmetic for attention); ``exact`` gives the same outputs from the definition
(64 bits for attention, row by row on the host for the bookkeeping). Sizes: 32 heads of
128 are the 4096 columns of the benchmark's projections; the rest is generic.

The bookkeeping is three int32 tensors: page_refs [pages] (how many places of the table
hold each page; 0: free), page_table [batch, width], kv_lens [batch]. A pass of one of
its operators begins by setting them back to the step's beginning (one copy of the flat
buffer that holds all three), so that every pass does the same work.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------- the cases
def _attention(name, batch, decoding, new, ctx, heads, kv_heads, dim, page, dtype, cap=0.0, distance=False, prefix=0,
               document=0, window=0, sinks=0, heads_first=False):
    return {"name": name, "op": "attention", "batch": batch, "decoding": decoding, "new": new, "ctx": ctx,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "type": dtype, "cap": cap,
            "distance": distance, "prefix": prefix, "document": document, "window": window, "sinks": sinks,
            "heads_first": heads_first}


def _copy(name, pairs, skipped, caches, pages, page, kv_heads, dim, heads_first, dtype):
    return {"name": name, "op": "copy", "pairs": pairs, "skipped": skipped, "caches": caches, "pages": pages,
            "page": page, "kv_heads": kv_heads, "dim": dim, "heads_first": heads_first, "type": dtype}


def _book(name, op, batch, ctx, page, beams, spare, **kw):
    """beams: rows to a group that share pages; spare: free pages for each used one."""
    return {"name": name, "op": op, "batch": batch, "ctx": ctx, "page": page, "beams": beams, "spare": spare} | kw


def listed():
    return [
        # one token of one sequence, heads that forget with distance, one K/V head for each query head: latency only
        _attention("decode_distance", 1, 1, 1, 1037, 32, 32, 128, 16, "f16", distance=True),
        # a serving step of a model with capped scores: 64 sequences of unlike lengths, 4 query heads to a K/V head
        _attention("decode_capped", 64, 64, 1, 8192, 32, 8, 128, 16, "bf16", cap=50.0),
        # 4096 new tokens on top of 12288 with capped scores: the arithmetic of a long prompt
        _attention("chunk_capped", 1, 0, 4096, 16384, 32, 8, 128, 64, "f16", cap=30.0),
        # prompts of several documents each, the first with a part that is seen both ways; odd lengths
        _attention("prompt_documents", 3, 0, 2500, 2500, 32, 8, 128, 32, "bf16", distance=True, prefix=577, document=700,
                   heads_first=True),
        # the last pages of four sequences that were forked, in K and V of 32 layers
        _copy("copy_forked", 4, 0, 64, 96, 16, 8, 128, False, "bf16"),
        # what a defragmentation moves: a list that is half filled, large pages, heads before positions
        _copy("copy_moved", 500, 524, 16, 1400, 64, 8, 64, True, "f16"),
        # beam search: 16 groups of 4 beams, each beam continued from one of its group
        _book("fork_beams", "fork", 64, 4000, 16, 4, 0.3, restarts=False),
        # 512 samples of long prompts, half of them restarted from another one of 16
        _book("fork_samples", "fork", 512, 30000, 16, 16, 0.2, restarts=True),
        # a decoding step of 61 sequences just forked in pairs: a token each, shared last pages replaced
        _book("append_step", "append", 62, 3000, 16, 2, 0.2, new=1, accepted=0),
        # drafts and prompts: 256 sequences take up to 1000 positions and give half of them back
        _book("append_drafts", "append", 256, 20000, 32, 1, 1.5, new=1000, accepted=1),
        # a small pool at the end of a burst
        _book("compact_small", "compact", 16, 4000, 16, 1, 1.0, moves=256),
        # a pool of half a million pages, three quarters of them free
        _book("compact_large", "compact", 256, 16384, 16, 2, 3.0, moves=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["decode", "decode", "chunk", "chunk", "mixed", "copy", "fork", "append", "compact"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128, 128, rng.choice([72, 80, 96, 112])])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if kind == "copy":
        pairs, caches = _log(rng, 1, 600), _log(rng, 1, 64)
        pairs = max(1, min(pairs, int(5e8 / (caches * page * kv_heads * dim * 2))))
        return _copy("copy", pairs, rng.choice([0, pairs, 3 * pairs + 1]), caches, 2 * pairs + rng.randrange(1, 60), page,
                     kv_heads, dim, rng.random() < 0.5, dtype)
    if kind in ("fork", "append", "compact"):
        batch = _log(rng, 1, 512)
        ctx = _log(rng, 1, min(60000, 10000000 // batch))
        beams = rng.choice([1, 2, 3, 4, 8])
        if kind == "fork":
            return _book("fork", "fork", batch, ctx, page, max(2, beams), rng.uniform(0, 1), restarts=rng.random() < 0.3)
        if kind == "append":
            return _book("append", "append", batch, ctx, page, beams, rng.uniform(0.02, 2), new=_log(rng, 1, 2000),
                         accepted=rng.choice([0, 1]))
        return _book("compact", "compact", batch, ctx, page, beams, rng.uniform(0, 4), moves=_log(rng, 1, 10000))
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    forms = {"cap": rng.choice([0.0, 20.0, 30.0, 50.0]), "distance": rng.random() < 0.5}
    forms["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    forms["sinks"] = rng.choice([0, 4, 37]) if forms["window"] else 0
    forms["heads_first"] = rng.random() < 0.5
    if kind == "decode":
        ctx = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(128, (1 << 22) // (ctx * kv_heads))))
        forms["document"] = rng.choice([0, 0, _log(rng, 20, 5000)])
        return _attention("decode", batch, batch, 1, ctx, heads, kv_heads, dim, page, dtype, **forms)
    new = _log(rng, 2, 3000)
    ctx = max(new, rng.choice([new, _log(rng, 2, 16000)]))
    forms["document"] = rng.choice([0, _log(rng, 20, 5000)])
    forms["prefix"] = rng.choice([0, _log(rng, 1, ctx)])
    batch = max(1, min(_log(rng, 1, 32), int(4.0e8 / (new * ctx * heads)), int(1.5e6 / (ctx * kv_heads))))
    decoding = batch - 1 if kind == "mixed" else 0
    return _attention(kind, batch, decoding, new, ctx, heads, kv_heads, dim, page, dtype, **forms)


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


def _document_starts(case, n, kv):
    """Where the documents of a sequence's last n positions begin: documents of unlike lengths, one after another."""
    ends, at, i = [], 0, 0
    while case["document"] and at < kv:
        at += max(1, int(case["document"] * (1.0, 0.4, 1.7, 0.05)[i % 4]))
        i += 1
        ends.append(at)
    pos = np.arange(kv - n, kv)
    begins = np.array([0] + ends)
    return begins[np.searchsorted(begins, pos, side="right") - 1]


def _prefixes(case):
    return [int(case["prefix"] * (1.0 - 0.3 * (i % 3))) for i in range(case["batch"])]


def _slopes(heads):
    """A geometric run from 2^(-8 / heads) to 2^-8."""
    return [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]


# ----------------------------------------------------------------- the bookkeeping of a case
def _rows(case):
    """(lengths, groups): the positions of each row, and the row that its shared pages come from."""
    b, w = case["batch"], case["beams"]
    lens, leader = [], []
    for i in range(b):
        first = i // w * w
        share = 1.0 - 0.75 * ((first * 7919) % b) / b
        n = max(1, int(case["ctx"] * share))
        # rows that were just forked are alike; others have gone on on their own for a while
        lens.append(n if case["op"] == "append" else n + (i - first) * 3)
        leader.append(first)
    return lens, leader


def _parents(case):
    """Which row each one goes on from: any of its group, or (restarts) every second one from another, the others from themselves."""
    b, w = case["batch"], case["beams"]
    if case["restarts"]:
        return [i // w * w + (i * 5 + 3) % w if i % 2 and i // w * w + w <= b else i for i in range(b)]
    out = []
    for i in range(b):
        first = i // w * w
        out.append(first + (i * i + 1) % min(w, b - first))
    return out


def _new_tokens(case):
    """New positions of each row: all take one, or every fourth a share of a prompt and the others a few."""
    if case["new"] == 1:
        return [0 if i % 31 == 30 else 1 for i in range(case["batch"])]
    return [case["new"] - (i * 37) % (case["new"] // 2 + 1) if i % 4 == 0 else min(case["new"], 1 + i % 8)
            for i in range(case["batch"])]


def _kept(case, lens, new):
    """Lengths that the rows are cut to after an append: half of what they took, or nothing (every seventh row ends)."""
    return [0 if i % 7 == 6 else n + (k // 2 if case["accepted"] else k) for i, (n, k) in enumerate(zip(lens, new))]


def _width(case):
    lens, _ = _rows(case)
    page = case["page"]
    return max(-(-n // page) for n in lens) + (-(-case["new"] // page) + 1 if case["op"] == "append" else 2)


def _pool(case):
    """(places in the table that are used, distinct used pages, pages in all)"""
    lens, leader = _rows(case)
    page = case["page"]
    held = sum(-(-n // page) for n in lens)
    distinct = 0
    for i, n in enumerate(lens):
        distinct += -(-n // page) - (_shared(case, lens, i, leader[i]) if leader[i] != i else 0)
    return held, distinct, distinct + int(distinct * case["spare"]) + 1


def _shared(case, lens, i, first):
    """Pages that row i has in common with its group's first row: all of them just after a fork, else three quarters."""
    if case["op"] == "append":
        return -(-lens[i] // case["page"])
    return lens[first] // case["page"] * 3 // 4


def _build(case, seed):
    """numpy (refs, table, lens) of the step's beginning; which pages are whose follows the seed."""
    rng = np.random.default_rng(seed)
    lens, leader = _rows(case)
    pages = _pool(case)[2]
    order = rng.permutation(pages).astype(np.int32)
    table = rng.integers(0, pages, (case["batch"], _width(case)), dtype=np.int32)       # unused places hold anything
    refs = np.zeros(pages, dtype=np.int32)
    at = 0
    for i, n in enumerate(lens):
        count = -(-n // case["page"])
        same = _shared(case, lens, i, leader[i]) if leader[i] != i else 0
        table[i, :same] = table[leader[i], :same]
        table[i, same:count] = order[at:at + count - same]
        at += count - same
        np.add.at(refs, table[i, :count], 1)
    return refs, table, np.array(lens, dtype=np.int32)


# ----------------------------------------------------------------- the inputs
def _normal(gen, shape, dtype):
    return torch.randn(shape, device="cuda", generator=gen).to(dtype)


def _int32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _cache(gen, case, pages, dtype):
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    if case["heads_first"]:
        return _normal(gen, (pages, hk, page, d), dtype).transpose(1, 2)
    return _normal(gen, (pages, page, hk, d), dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "copy":
        s["caches"] = [_cache(gen, case, case["pages"], TYPES[case["type"]]) for _ in range(case["caches"])]
        order = torch.randperm(case["pages"], device="cuda", generator=gen)[:2 * case["pairs"]].to(torch.int32)
        none = torch.full((case["skipped"],), -1, dtype=torch.int32, device="cuda")
        s["src"], s["dst"] = torch.cat((order[:case["pairs"]], none)), torch.cat((order[case["pairs"]:], none))
        return s
    if case["op"] != "attention":
        refs, table, lens = _build(case, seed)
        s["start"] = _int32(np.concatenate((refs, lens, table.ravel())))
        s["flat"] = s["start"].clone()
        n, b = len(refs), case["batch"]
        s["page_refs"], s["kv_lens"] = s["flat"][:n], s["flat"][n:n + b]
        s["page_table"] = s["flat"][n + b:].view(b, -1)
        if case["op"] == "fork":
            s["parents"] = _int32(_parents(case))
        if case["op"] == "append":
            new = _new_tokens(case)
            s["q_starts"], s["tokens"] = _int32(np.concatenate(([0], np.cumsum(new)))), sum(new)
            s["kept"] = _int32(_kept(case, lens, new))
        return s
    dtype, d = TYPES[case["type"]], case["dim"]
    new, kv = _lengths(case)
    page = case["page"]
    per = [-(-n // page) for n in kv]
    pages = sum(per) + 2
    s["k_cache"], s["v_cache"] = _cache(gen, case, pages, dtype), _cache(gen, case, pages, dtype)
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.zeros((case["batch"], max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    s["page_table"], s["kv_lens"] = table, _int32(kv)
    s["q_starts"], s["max_new"] = _int32(np.concatenate(([0], np.cumsum(new)))), max(new)
    # queries of several lengths: scores from well below the cap to several times it
    q = torch.randn((sum(new), case["heads"], d), device="cuda", generator=gen)
    q *= torch.linspace(0.5, 3.0 if not case["cap"] else 0.5 * case["cap"], case["heads"], device="cuda")[None, :, None]
    s["q"], s["scale"] = q.to(dtype), 1.0 / math.sqrt(d)
    s["slopes"] = torch.tensor(_slopes(case["heads"]), device="cuda") if case["distance"] else None
    s["prefix_lens"] = _int32(_prefixes(case)) if case["prefix"] else None
    s["doc_starts"] = None
    if case["document"]:
        s["doc_starts"] = _int32(np.concatenate([_document_starts(case, n, k) for n, k in zip(new, kv)]))
    if own:
        from qkv_projection_gb300 import kaio
        s["workspace"] = kaio.paged_attention_workspace()
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    if "flat" in state:
        state["flat"].copy_(state["start"])
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"attention": _plain_attention, "copy": _plain_copy, "fork": _plain_fork, "append": _plain_append,
            "compact": _plain_compact}[op](state)


def _book_state(s):
    return {"page_refs": s["page_refs"], "page_table": s["page_table"], "kv_lens": s["kv_lens"]}


def _run_own(s, op):
    from qkv_projection_gb300 import kaio
    c = s["case"]
    if op == "attention":
        out, lse = kaio.paged_attention(
            s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_starts"], max_new=s["max_new"],
            scale=s["scale"], window=c["window"], sinks=c["sinks"], workspace=s["workspace"], return_lse=True,
            softcap=c["cap"], slopes=s["slopes"], prefix_lens=s["prefix_lens"], doc_starts=s["doc_starts"])
        return {"out": out, "lse": lse}
    if op == "copy":
        kaio.cache_copy_pages(s["caches"], s["src"], s["dst"])
        return list(s["caches"])
    book = (s["page_refs"], s["page_table"], s["kv_lens"])
    if op == "fork":
        kaio.cache_fork(*book, s["parents"], c["page"])
        return _book_state(s)
    if op == "append":
        slots, src, dst = kaio.cache_append(*book, s["q_starts"], s["tokens"], c["page"])
        kaio.cache_truncate(*book, s["kept"], c["page"])
        return _book_state(s) | {"slots": slots, "src": src, "dst": dst}
    src, dst = kaio.cache_compact(*book, c["page"], c["moves"])
    return _book_state(s) | {"src": src, "dst": dst}


def _plain_copy(s):
    real = s["src"] >= 0
    pairs = s["case"]["pairs"]                                 # the real ones come first
    src, dst = s["src"][:pairs].long(), s["dst"][:pairs].long()
    real = real[:pairs, None, None, None]
    for cache in s["caches"]:
        cache[dst] = torch.where(real, cache[src], cache[dst])
    return list(s["caches"])


def _ceil(x, page):
    return torch.div(x + (page - 1), page, rounding_mode="floor")


def _count(refs, pages, held, by):
    """Adds `by` to the references of those `pages` that are `held`."""
    n = refs.numel()
    more = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    more.index_add_(0, torch.where(held, pages.long(), n).flatten(),
                    torch.full((pages.numel(),), by, dtype=torch.int32, device="cuda"))
    refs += more[:n]


def _plain_fork(s):
    refs, table, lens, page = s["page_refs"], s["page_table"], s["kv_lens"], s["case"]["page"]
    parents = s["parents"].long()
    place = torch.arange(table.shape[1], device="cuda")
    changed = (parents != torch.arange(len(parents), device="cuda"))[:, None]
    held = (place < _ceil(lens, page)[:, None]) & changed
    new_lens = lens[parents]
    new_held = (place < _ceil(new_lens, page)[:, None]) & changed
    new = table[parents]
    _count(refs, table, held, -1)
    _count(refs, new, new_held, 1)
    table.copy_(torch.where(new_held, new, table))
    lens.copy_(new_lens)
    return _book_state(s)


def _plain_append(s):
    refs, table, lens, page = s["page_refs"], s["page_table"], s["kv_lens"], s["case"]["page"]
    n, (batch, width) = refs.numel(), table.shape
    starts = s["q_starts"].long()
    new, old = starts[1:] - starts[:-1], lens.long()
    have, want = _ceil(old, page), _ceil(old + new, page)
    fits = old + new <= width * page
    last = (have - 1).clamp(min=0)
    last_page = table.gather(1, last[:, None])[:, 0].long()
    tail = (new > 0) & (old % page != 0) & (refs[last_page.clamp(0, n - 1)] > 1)
    need = torch.where(fits & (new > 0), want - have + tail, 0)
    before = torch.cumsum(need, 0) - need
    free = refs <= 0
    order = torch.argsort((~free).to(torch.uint8), stable=True)                    # free pages first, the lowest first
    granted = fits & (new > 0) & ((need == 0) | (before + need <= free.sum()))
    tail &= granted
    first = order[before.clamp(max=n - 1)]
    src, dst = torch.where(tail, last_page, -1), torch.where(tail, first, -1)
    place = torch.arange(width, device="cuda")
    fresh = granted[:, None] & (place >= have[:, None]) & (place < want[:, None])
    taken = order[(before + tail - have)[:, None].add(place).clamp(0, n - 1)]
    table.copy_(torch.where(fresh, taken, table))
    table.copy_(torch.where(tail[:, None] & (place == last[:, None]), first[:, None], table))
    _count(refs, last_page, tail, -1)
    _count(refs, first, tail, 1)
    _count(refs, taken, fresh, 1)
    lens.copy_(torch.where(granted, old + new, old))
    t = torch.arange(s["tokens"], device="cuda")
    row = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    at = old[row] + t - starts[row]
    got = table[row, torch.div(at, page, rounding_mode="floor").clamp(max=width - 1)].long()
    slots = torch.where(granted[row], got * page + at % page, -1)
    # the cut
    kept = torch.minimum(lens, s["kept"])
    gone = (place >= _ceil(kept, page)[:, None]) & (place < _ceil(lens, page)[:, None])
    _count(refs, table, gone, -1)
    lens.copy_(kept)
    return _book_state(s) | {"slots": slots.int(), "src": src.int(), "dst": dst.int()}


def _plain_compact(s):
    refs, table, lens, page = s["page_refs"], s["page_table"], s["kv_lens"], s["case"]["page"]
    n, moves = refs.numel(), min(s["case"]["moves"], refs.numel())
    free = refs <= 0
    low = torch.argsort((~free).to(torch.uint8), stable=True)[:moves]              # free pages, the lowest first
    high = (n - 1) - torch.argsort(free.flip(0).to(torch.uint8), stable=True)[:moves]      # used ones, the highest first
    i = torch.arange(moves, device="cuda")
    ok = (low < high) & (i < free.sum()) & (i < n - free.sum())
    src = torch.full((s["case"]["moves"],), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[:moves], dst[:moves] = torch.where(ok, high, -1).int(), torch.where(ok, low, -1).int()
    to = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    to[torch.where(ok, high, n)] = torch.where(ok, low, n).int()
    place = torch.arange(table.shape[1], device="cuda")
    held = place < _ceil(lens, page)[:, None]
    table.copy_(torch.where(held, to[table.long()], table))
    moved = refs.clone()
    more = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    more[torch.where(ok, low, n)] = moved[high]
    less = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    less[torch.where(ok, high, n)] = moved[high]
    refs += more[:n] - less[:n]
    return _book_state(s) | {"src": src, "dst": dst}


def _plain_attention(s):
    c = s["case"]
    b, hk, d, n = c["batch"], c["kv_heads"], c["dim"], s["max_new"]
    group = c["heads"] // hk
    kv, starts = s["kv_lens"].long(), s["q_starts"].long()
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
    seen = j <= pos[:, :, None]
    if c["window"]:
        seen &= (j > pos[:, :, None] - c["window"]) | (j < c["sinks"])
    if c["prefix"]:
        seen |= j < s["prefix_lens"].long()[:, None, None]
    if c["document"]:
        seen &= j >= s["doc_starts"].long()[token][:, :, None]
    seen &= j < kv[:, None, None]
    score = torch.matmul(q, k).reshape(b, hk, group, n, width)
    score *= s["scale"]
    if c["cap"]:
        score.div_(c["cap"]).tanh_().mul_(c["cap"])
    if c["distance"]:
        apart = (pos[:, :, None] - j).abs().float()                                   # [b, n, width]
        slope = s["slopes"].reshape(hk, group, 1, 1)
        for at in range(b):
            score[at].sub_(slope * apart[at])
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
def _seen(case, n, kv, prefix):
    """(query-key pairs, distinct keys) that a sequence's n new tokens see."""
    p = np.arange(kv - n, kv, dtype=np.int64)
    ds = _document_starts(case, n, kv)
    hi = np.maximum(p + 1, min(prefix, kv))
    lo = np.maximum(p - case["window"] + 1, 0) if case["window"] else np.zeros_like(p)
    first = np.minimum(max(case["sinks"] if case["window"] else 0, prefix), hi)
    a = np.maximum(np.minimum(first, np.maximum(lo, ds)) - ds, 0)                     # the part before the run
    pairs = int((a + hi - np.maximum(lo, ds)).sum())
    marks = np.zeros(kv + 1, dtype=np.int64)
    for l0, h0 in ((ds, ds + a), (np.maximum(lo, ds), hi)):
        np.add.at(marks, l0, 1)
        np.add.at(marks, h0, -1)
    return pairs, int((np.cumsum(marks[:-1]) > 0).sum())


def work(case):
    if case["op"] == "copy":
        size = case["pairs"] * case["caches"] * case["page"] * case["kv_heads"] * case["dim"] * 2
        return {"bytes": 2 * size + 8 * (case["pairs"] + case["skipped"]), "flops": 0}
    if case["op"] == "attention":
        d = case["dim"]
        new, kv = _lengths(case)
        seen = [_seen(case, n, k, p) for n, k, p in zip(new, kv, _prefixes(case))]
        keys, pairs, tokens = sum(x[1] for x in seen), sum(x[0] for x in seen), sum(new)
        return {"bytes": 4 * tokens * case["heads"] * d + 4 * keys * case["kv_heads"] * d + 4 * tokens * case["heads"]
                + 4 * sum(-(-k // case["page"]) for k in kv) + 8 * case["batch"]
                + (4 * case["heads"] if case["distance"] else 0) + (4 * tokens if case["document"] else 0)
                + (4 * case["batch"] if case["prefix"] else 0),
                "flops": 4 * d * case["heads"] * pairs}
    lens, _ = _rows(case)
    page, b = case["page"], case["batch"]
    held, distinct, pages = _pool(case)
    if case["op"] == "fork":
        changed = [(i, p) for i, p in enumerate(_parents(case)) if i != p]
        entries = sum(2 * -(-lens[p] // page) + -(-lens[i] // page) for i, p in changed)
        return {"bytes": 4 * (entries + 3 * b) + 8 * distinct, "flops": entries}
    if case["op"] == "append":
        new = _new_tokens(case)
        taken = sum(-(-(n + k) // page) - -(-n // page) for n, k in zip(lens, new))
        return {"bytes": 4 * (pages + 2 * taken + 6 * b + 2 * b + sum(new)), "flops": pages}
    return {"bytes": 4 * (pages + held + 2 * case["moves"]), "flops": pages}


# ----------------------------------------------------------------- the definition
def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, seed)
    if case["op"] == "copy":
        s = prepare(case, seed)
        out = [c.clone() for c in s["caches"]]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for c in out if a >= 0 else ():
                c[b] = c[a]
        return out
    refs, table, lens = _build(case, seed)
    page = case["page"]
    refs, count = refs.tolist(), lambda n: -(-int(n) // page)  # noqa: E731
    more = {}
    if case["op"] == "fork":
        before, lens0 = table.copy(), lens.copy()
        for row, parent in enumerate(_parents(case)):
            if row == parent:
                continue
            for p in before[row, :count(lens0[row])]:
                refs[p] -= 1
            for p in before[parent, :count(lens0[parent])]:
                refs[p] += 1
            table[row, :count(lens0[parent])] = before[parent, :count(lens0[parent])]
            lens[row] = lens0[parent]
    elif case["op"] == "append":
        new = _new_tokens(case)
        free = [p for p, r in enumerate(refs) if r <= 0]
        shared = [r > 1 for r in refs]
        at, slots, src, dst, old = 0, [], [-1] * len(new), [-1] * len(new), lens.tolist()
        for row, n in enumerate(new):
            have, want = count(old[row]), count(old[row] + n)
            tail = n > 0 and old[row] % page != 0 and shared[table[row, have - 1]]
            need = want - have + tail
            if n == 0 or old[row] + n > table.shape[1] * page or (need and at + need > len(free)):
                slots += [-1] * n
                at += need if n and old[row] + n <= table.shape[1] * page else 0
                continue
            mine = free[at:at + need]
            at += need
            if tail:
                src[row], dst[row] = int(table[row, have - 1]), mine[0]
                refs[src[row]] -= 1
                table[row, have - 1] = mine[0]
            table[row, have:want] = mine[int(tail):]
            for p in mine:
                refs[p] += 1
            slots += [int(table[row, k // page]) * page + k % page for k in range(old[row], old[row] + n)]
            lens[row] += n
        for row, n in enumerate(_kept(case, old, new)):
            if n < lens[row]:
                for p in table[row, count(n):count(lens[row])]:
                    refs[p] -= 1
                lens[row] = n
        more = {"slots": slots, "src": src, "dst": dst}
    else:
        src, dst = [-1] * case["moves"], [-1] * case["moves"]
        low, high, to = 0, len(refs) - 1, {}
        for i in range(case["moves"]):
            while low < len(refs) and refs[low] > 0:
                low += 1
            while high >= 0 and refs[high] <= 0:
                high -= 1
            if low >= high:
                break
            src[i], dst[i], to[high] = high, low, low
            refs[low], refs[high] = refs[high], 0
        for row in range(len(lens)):
            n = count(lens[row])
            table[row, :n] = [to.get(p, p) for p in table[row, :n].tolist()]
        more = {"src": src, "dst": dst}
    return {k: _int32(v) for k, v in (dict(page_refs=refs, page_table=table, kv_lens=lens) | more).items()}


def _exact_attention(case, seed):
    s = prepare(case, seed)
    new, kv = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    slopes = torch.tensor(_slopes(case["heads"]), device="cuda").double()              # as the f32 that they are
    row = 0
    for b, (n, length, prefix) in enumerate(zip(new, kv, _prefixes(case))):
        count = -(-length // case["page"])
        ids = s["page_table"][b, :count].long()
        keys = s["k_cache"][ids].flatten(0, 1)[:length]
        values = s["v_cache"][ids].flatten(0, 1)[:length]
        ds = torch.tensor(_document_starts(case, n, length), device="cuda")
        j = torch.arange(length, device="cuda")
        step = max(1, (1 << 26) // (length * group))
        for h in range(case["kv_heads"]):
            kh, vh = keys[:, h].double(), values[:, h].double()
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                p = torch.arange(length - n + i0, length - n + i1, device="cuda")[:, None]
                hidden = j > p
                if case["window"]:
                    hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
                hidden = (hidden & (j >= prefix)) | (j < ds[i0:i1, None])
                rows, heads = slice(row + i0, row + i1), slice(h * group, (h + 1) * group)
                x = torch.einsum("igd,jd->igj", s["q"][rows, heads].double(), kh) * s["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["distance"]:
                    x = x - slopes[heads][None, :, None] * (p - j).abs()[:, None, :]
                x = x.masked_fill(hidden[:, None, :], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[rows, heads] = z
                out[rows, heads] = torch.einsum("igj,jd->igd", torch.exp(x - z[..., None]), vh)
        row += n
    return {"out": out, "lse": lse}
