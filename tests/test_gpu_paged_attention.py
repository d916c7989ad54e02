"""Attention over a paged cache against the 64-bit definition.

Tolerance, per output value, with u = 2^-p of the tensors' type (p = 11 or 8
significant bits), A = sum_j p_j |v_j| and S = |scale| max_j sum_d |q_d k_jd|
from the definition:
- the result is rounded once: u * |out| (and 2^-25, half the smallest f16 subnormal);
- each weight is rounded to the type before the second product, its sum is not: u * A;
- scores are f32 sums of d products: off by at most d * 2^-24 * S, and the scale,
  the exponent's argument and the exponential itself by a few 2^-24 * (S + 1); a
  score off by e changes a weight by e relative, twice (weight and sum): 2 e A;
- sums over the keys in f32, in pieces of at most a few thousand: 2^-24 * keys / 4
  would be the worst case of a piece; 1e-5 * A covers pieces of 600 keys at their
  worst and any length as a random walk.
lse: e + 1e-5 * (1 + |lse|).
"""
import numpy as np
import pytest

from oracle.attention import paged_attention_ref
from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu

BITS = {"float16": 11, "bfloat16": 8}


class Problem:
    """lens: (new tokens, cache positions) of each sequence."""

    def __init__(self, lens, heads=4, kv_heads=2, d=64, page=16, dtype="float16", layout="slots_first", seed=0,
                 extra_pages=1, extra_table=0, spread=1.5):
        import torch
        self.dtype, self.d, self.page, self.heads, self.kv_heads = dtype, d, page, heads, kv_heads
        td = getattr(torch, dtype)
        g = torch.Generator(device="cuda").manual_seed(seed)
        per = [-(-kv // page) for _, kv in lens]
        pages = sum(per) + extra_pages
        if layout == "heads_first":
            kc, vc = (torch.randn(pages, kv_heads, page, d, device="cuda", generator=g).to(td).transpose(1, 2)
                      for _ in range(2))
        elif layout == "one_buffer":
            both = torch.randn(pages, 2, page, kv_heads, d, device="cuda", generator=g).to(td)
            kc, vc = both[:, 0], both[:, 1]
        else:
            kc, vc = (torch.randn(pages, page, kv_heads, d, device="cuda", generator=g).to(td) for _ in range(2))
        self.kc, self.vc = kc, vc
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        table = torch.full((len(lens), max(max(per), 1) + extra_table), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.lens = lens
        self.kv = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
        starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.q = (torch.randn(int(starts[-1]), heads, d, device="cuda", generator=g) * spread).to(td)
        self.scale = d ** -0.5

    def run(self, **kw):
        kw.setdefault("q_starts", self.starts)
        kw.setdefault("max_new", max(n for n, _ in self.lens))
        kw.setdefault("return_lse", True)
        return kaio.paged_attention(kw.pop("q", self.q), self.kc, self.vc, self.table, self.kv, **kw)

    def ref(self, causal=True, window=0, sinks=0, scale=None):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        return paged_attention_ref(f(self.q), f(self.kc), f(self.vc), self.table.cpu().numpy(),
                                   self.kv.tolist(), self.starts.tolist(), self.scale if scale is None else scale,
                                   causal, window, sinks)

    def check(self, got, ref):
        out, lse = (t.double().cpu().numpy() for t in got)
        want, want_lse, spread, size = ref
        u = 2.0 ** -BITS[self.dtype]
        e = (self.d + 8) * 2.0 ** -24 * (size + 1)
        bound = u * np.abs(want) + (u + 2 * e[..., None] + 1e-5) * spread + 2.0 ** -25
        err = np.abs(out - want)
        assert np.all(err <= bound), ((err - bound).max(), np.argwhere(~(err <= bound))[:4])
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(lse), none) and not out[none].any()
        le = np.abs(lse[~none] - want_lse[~none])
        assert np.all(le <= e[~none] + 1e-5 * (1 + np.abs(want_lse[~none]))), le.max()

    def verify(self, **mask):
        got = self.run(**mask)
        self.check(got, self.ref(**mask))
        return got


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kv_heads,d,page,layout", [
    (4, 4, 128, 16, "slots_first"), (8, 2, 64, 32, "heads_first"), (15, 3, 72, 64, "one_buffer"),
    (7, 1, 96, 128, "slots_first"), (16, 1, 128, 1024, "heads_first"), (40, 2, 8, 16, "slots_first"),
])
def test_single_tokens(heads, kv_heads, d, page, layout, dtype):
    lens = [(1, n) for n in (1, 16, 0, 17, 63, 64, 65, 129, 1000, 0, 2311)]
    p = Problem(lens, heads, kv_heads, d, page, dtype, layout, seed=heads)
    got = p.verify()
    again = kaio.paged_attention(p.q, p.kc, p.vc, p.table, p.kv, return_lse=True)     # one token each, by default
    assert all((a == b).all() for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kv_heads,d,page,lens", [
    (4, 4, 128, 16, [(130, 130)]),
    (8, 2, 128, 16, [(5, 300), (0, 77), (64, 64), (1, 500), (33, 129)]),
    (6, 3, 64, 32, [(257, 700)]),
    (5, 1, 80, 64, [(100, 333), (2, 2), (40, 41)]),
    (7, 1, 112, 128, [(19, 150), (1, 1), (75, 1025)]),
    (2, 2, 16, 16, [(300, 300), (0, 0), (127, 128)]),
    (24, 1, 64, 256, [(3, 1000), (12, 700), (1, 2000)]),
])
def test_chunks(heads, kv_heads, d, page, lens, dtype):
    Problem(lens, heads, kv_heads, d, page, dtype, seed=d).verify()


@pytest.mark.parametrize("lens", [
    [(4, 0)], [(5, 2)], [(200, 100), (1, 1)], [(300, 7), (2, 900)], [(0, 0), (3, 3)],
])
def test_rows_that_see_nothing(lens):
    """More new tokens than positions: the first ones stand before the cache's start."""
    for d in (64, 128):
        Problem(lens, 6, 2, d).verify()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (37, 70), (128, 4), (100, 128), (700, 33),
                                          (5000, 4), (64, 5000), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("lens", [[(1, 700), (1, 3), (1, 130)], [(90, 1000), (3, 3), (1, 64)], [(400, 640)]])
def test_window_and_sinks(lens, window, sinks):
    p = Problem(lens, 4, 2, 64, 16, seed=window % 1000)
    p.verify(window=window, sinks=sinks)


def test_window_at_full_width():
    Problem([(1, 4000), (300, 3001), (7, 7)], 8, 2, 128, 32, "bfloat16").verify(window=512, sinks=5)


@pytest.mark.parametrize("lens", [[(1, 200), (1, 0)], [(70, 300), (5, 2)], [(150, 150)]])
def test_without_causal_order(lens):
    p = Problem(lens, 4, 1, 128)
    p.verify(causal=False)
    p.verify(causal=False, window=40, sinks=3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    for lens in ([(1, 300)], [(140, 300)]):
        p = Problem(lens, 2, 2, 128)
        p.check(p.run(scale=scale), p.ref(scale=scale))


def test_scores_that_rise_and_fall_along_the_keys():
    """The running maximum has to be renewed often, and by a lot."""
    import torch
    for n in (1, 200):
        p = Problem([(n, 900)], 2, 1, 64, 16)
        ramp = torch.cat((torch.linspace(-40, 60, 450), torch.linspace(60, -300, 450))).cuda()
        p.q[..., 0] = 8.0
        for j in range(900):
            p.kc[p.table[0, j // 16], j % 16, :, 0] = ramp[j].half()
        p.verify()


@pytest.mark.parametrize("lens,mask", [
    ([(1, 501)], {}), ([(1, 3000)], dict(window=200, sinks=20)), ([(100, 2000)], dict(window=300, sinks=3)),
    ([(200, 777), (1, 45)], {}),
])
def test_what_no_token_sees_may_hold_anything(lens, mask):
    """NaN, infinities and the type's lowest value in slots that no new token sees;
    table entries of such pages far outside the cache."""
    import torch
    p = Problem(lens, 4, 2, 128, 16, extra_pages=4, extra_table=3, seed=8)
    ref = p.ref(**mask)
    seen = torch.zeros(p.kc.shape[:2], dtype=torch.bool, device="cuda")
    bad = torch.tensor([2**31 - 1, -1, -2**31, p.kc.shape[0]], dtype=torch.int32, device="cuda")
    for b, (n, kv) in enumerate(lens):
        lo = max(0, kv - n - mask["window"] + 1) if mask else 0
        for j in range(kv):
            if j >= lo or j < mask.get("sinks", 0):
                seen[p.table[b, j // 16], j % 16] = True
        for i in range(p.table.shape[1]):
            first, past = i * 16, i * 16 + 16
            if first >= kv or (past <= lo and first >= mask.get("sinks", 0)):
                p.table[b, i] = bad[i % 4]
    junk = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float16).min],
                        dtype=torch.float16, device="cuda")
    for c in (p.kc, p.vc):
        c[~seen] = junk[torch.arange(p.d, device="cuda") % 4].expand(int((~seen).sum()), p.kv_heads, p.d)
    p.check(p.run(**mask), ref)


def test_pages_outside_the_cache_read_as_zeros():
    import torch
    for n in (1, 40):
        p = Problem([(n, 200)], 4, 2, 64, 16)
        page = int(p.table[0, 3])
        p.kc[page] = 0
        p.vc[page] = 0
        want = p.run()
        for bad in (-1, p.kc.shape[0], 2**31 - 1):
            p.table[0, 3] = bad
            assert all(torch.equal(a, b) for a, b in zip(want, p.run()))


def test_lengths_past_the_table_are_cut():
    import torch
    for n in (1, 30):
        p = Problem([(n, 160)], 4, 2, 64, 16)
        want = p.run()
        p.kv[0] = 100000
        assert all(torch.equal(a, b) for a, b in zip(want, p.run()))


@pytest.mark.parametrize("n", [1, 20])
def test_a_long_cache_past_32_bit_offsets(n):
    """Pages beyond 2^31 elements of the cache (4.3 GB), by either of the two strides."""
    import torch
    pages, page, kh, d = 18000, 64, 16, 128                         # 2.36e9 elements
    for first in (False, True):
        shape = (pages, kh, page, d) if first else (pages, page, kh, d)
        p = Problem([(n, 300)], 32, kh, d, page)
        small_k, small_v, small_t = p.kc, p.vc, p.table.clone()
        ref = p.ref()
        for name, small in (("kc", small_k), ("vc", small_v)):
            big = torch.empty(shape, dtype=torch.float16, device="cuda")
            big = big.transpose(1, 2) if first else big
            big[pages - small.shape[0]:] = small
            setattr(p, name, big)
        p.table = small_t + (pages - small_k.shape[0])
        p.check(p.run(), ref)


def test_long_context_is_split_and_joined_the_same_way_every_time():
    import torch
    for lens in ([(1, 30011)], [(20, 20000)], [(1, 9000), (1, 100), (64, 7000)]):
        p = Problem(lens, 8, 2, 64, 64)
        ws = kaio.paged_attention_workspace()
        first = p.run(workspace=ws)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, p.run(workspace=ws)))
        if sum(n for n, _ in lens) == 1:
            p.check(first, p.ref())


def test_many_sequences():
    p = Problem([(1 + i % 3 if i % 5 else 0, 3 + 7 * (i % 41)) for i in range(700)], 4, 2, 32, 16)
    p.verify()


def test_strided_queries_outputs_and_other_stream():
    import torch
    for n in (1, 77):
        p = Problem([(n, 150), (n, 90)], 6, 2, 64)
        want = p.verify()
        packed = torch.zeros(2 * n, 10, 64, dtype=torch.float16, device="cuda")     # q beside k and v
        packed[:, 2:8] = p.q
        out = torch.zeros(6, 2 * n, 64, dtype=torch.float16, device="cuda").transpose(0, 1)
        lse = torch.empty(2 * n, 6, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = p.run(q=packed[:, 2:8], out=out, lse=lse, stream=side)
        side.synchronize()
        assert got[0] is out and got[1] is lse
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(p.run(return_lse=False), want[0])


def test_in_a_graph():
    import torch
    for n in (1, 40):
        p = Problem([(n, 500)], 8, 2, 128)
        ws = kaio.paged_attention_workspace()
        out = torch.empty_like(p.q)
        want = p.run(workspace=ws, out=out)[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.run(workspace=ws, out=out, return_lse=False)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_nothing_to_do():
    import torch
    p = Problem([(0, 5), (0, 0)], 4, 2, 64)
    out, lse = p.run(max_new=0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # an empty cache: every token sees nothing
    q = torch.randn(2, 4, 64, device="cuda").half()
    cache = torch.empty(0, 16, 2, 64, dtype=torch.float16, device="cuda")
    table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    out, lse = kaio.paged_attention(q, cache, cache, table, torch.tensor([0, 9], dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    assert not out.any() and (lse == -float("inf")).all()


def test_refusals():
    import torch
    p = Problem([(1, 20)], 4, 2, 64)
    ok = lambda **kw: p.run(**kw)  # noqa: E731
    ok()
    for match, kw in (("window", dict(window=-1)), ("sinks", dict(sinks=-1)), ("scale", dict(scale=float("nan"))),
                      ("max_new", dict(max_new=-1)), ("overlaps input", dict(out=p.q)),
                      ("workspace_bytes", dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(kaio.KaioError, match=match):
            ok(**kw)
    with pytest.raises(ValueError, match="workspace"):
        ok(workspace=torch.zeros(64, device="cuda"))
    with pytest.raises(kaio.KaioError, match="without q_starts"):
        kaio.paged_attention(p.q.repeat(2, 1, 1), p.kc, p.vc, p.table, p.kv)
    with pytest.raises(kaio.KaioError, match="page_size"):
        kaio.paged_attention(p.q, p.kc[:, :12], p.vc[:, :12], p.table, p.kv)
    with pytest.raises(kaio.KaioError, match="multiple of kv_heads"):
        kaio.paged_attention(p.q[:, :3], p.kc, p.vc, p.table, p.kv)
    wide = torch.zeros(3, 16, 2, 136, dtype=torch.float16, device="cuda")
    with pytest.raises(kaio.KaioError, match="dim"):
        kaio.paged_attention(torch.zeros(1, 4, 136, dtype=torch.float16, device="cuda"), wide, wide, p.table, p.kv)
    with pytest.raises(TypeError, match="v_cache"):
        kaio.paged_attention(p.q, p.kc, p.vc.float(), p.table, p.kv)
    with pytest.raises(ValueError, match="v_cache"):
        kaio.paged_attention(p.q, p.kc, p.vc[:1], p.table, p.kv)
    with pytest.raises(TypeError, match="kv_lens"):
        kaio.paged_attention(p.q, p.kc, p.vc, p.table, p.kv.long())
    with pytest.raises(ValueError, match="page_table"):
        kaio.paged_attention(p.q, p.kc, p.vc, p.table[:0], p.kv)
    with pytest.raises(ValueError, match="dense last"):
        kaio.paged_attention(p.q.transpose(1, 2).contiguous().transpose(1, 2), p.kc, p.vc, p.table, p.kv)
    with pytest.raises(ValueError, match="gradient"):
        kaio.paged_attention(p.q.clone().requires_grad_(), p.kc, p.vc, p.table, p.kv)


def test_a_nan_query_or_key_stays_with_those_that_use_it():
    import torch
    for n in (1, 50):
        p = Problem([(n, 120), (n, 120)], 4, 2, 64)
        ref = p.ref()
        p.q[0, 1, 5] = float("nan")
        p.kc[p.table[1, 0], 3, 1, 7] = float("nan")            # second sequence, second K/V head
        out, lse = p.run()
        gone = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
        gone[0, 1] = True
        gone[n:, 2:] = True
        assert out[gone].isnan().all() and lse[gone].isnan().all()
        keep = (~gone).cpu().numpy()
        u = 2.0 ** -11
        err = (out.double().cpu().numpy() - ref[0])[keep]
        assert np.all(np.abs(err) <= (u * np.abs(ref[0]) + (u + 1e-4) * ref[2] + 2.0 ** -25)[keep])


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "float16")])
def test_tiles_of_one_half_between_tiles_of_two(d, dtype):
    """65 tokens of 4 heads are a tile of 256 rows and one of 4, over more key tiles than
    the shared memory holds at once, head after head and sequence after sequence."""
    Problem([(65, 2000), (1, 1500), (70, 1700), (33, 900), (64, 800)], 8, 2, d, 32, dtype).verify()


@pytest.mark.parametrize("n,kv", [(5, 129), (5, 256), (5, 257), (5, 384), (20, 1000), (32, 4000), (30, 40)])
def test_few_rows_of_a_chunk_share_the_keys_between_two_halves(n, kv):
    for mask in ({}, dict(window=100, sinks=3)):
        Problem([(n, kv), (n, kv - 3)], 8, 2, 128, 16, "bfloat16", seed=kv).verify(**mask)
        Problem([(n, kv), (0, 3), (n + 1, kv)], 4, 1, 64, 32, seed=n).verify(**mask)


def test_split_items_joined_by_whichever_part_comes_last():
    """The parts of an item that several CTAs share finish in any order; repeated calls
    go through all of the ways to join them."""
    import torch
    for args, lens in (((40, 2, 64, 16), [(1, 1000), (1, 2311)]), ((8, 1, 128, 32, "bfloat16"), [(64, 5000), (3, 900)])):
        p = Problem(lens, *args, seed=40)
        ws = kaio.paged_attention_workspace()
        first = p.verify()
        for _ in range(50):
            assert all(torch.equal(a, b) for a, b in zip(first, p.run(workspace=ws)))
