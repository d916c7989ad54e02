"""Attention with capped scores, a bias that grows with distance, documents and prefixes,
against the 64-bit definition.

Tolerance: that of test_gpu_paged_attention.py (its u, A and S), with a larger score error e:
- the slope of the tanh is at most one, so what scores are off before it is no larger after;
- the capped score is off by at most 24 * 2^-24 caps (the approximate exponential, its argument, the
  reciprocal and five roundings, times 2 caps; derived at cap4 in paged_chunk.cuh);
- the bias is slope * distance with three roundings (slope * log2(e), the product, the sum with the
  score) and, in chunks, up to sixteen additions of a step: 22 * 2^-24 of it for each key, which
  the weights p_j bound on average: far = sum_j p_j |bias_j|, farv = sum_j p_j |bias_j| |v_j|;
- the sum of the two is rounded: covered by the above and by e's (S + 1).
A weight off by e_j relative moves the output by sum_j p_j e_j |v_j| and, through the sum, by
sum_j p_j e_j * A.
"""
import numpy as np
import pytest

from qkv_projection_gb300 import kaio
from test_gpu_paged_attention import BITS, Problem

pytestmark = pytest.mark.gpu


class Scored(Problem):
    def ref(self, causal=True, window=0, sinks=0, scale=None, softcap=0.0, slopes=None, prefix_lens=None, doc_starts=None):
        from oracle.attention import paged_attention_ref
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        i = lambda t: None if t is None else t.tolist()  # noqa: E731
        self.far, self.cap = {}, softcap
        return paged_attention_ref(f(self.q), f(self.kc), f(self.vc), self.table.cpu().numpy(), self.kv.tolist(),
                                   self.starts.tolist(), self.scale if scale is None else scale, causal, window, sinks,
                                   softcap, None if slopes is None else f(slopes), i(prefix_lens), i(doc_starts), self.far)

    def check(self, got, ref):
        out, lse = (t.double().cpu().numpy() for t in got)
        want, want_lse, spread, size = ref
        u, f32 = 2.0 ** -BITS[self.dtype], 2.0 ** -24
        e = (self.d + 8) * f32 * (size + 1) + 24 * f32 * self.cap
        far, farv = self.far.get("b", np.zeros(size.shape)), self.far.get("bv", np.zeros(spread.shape))
        bound = (u * np.abs(want) + (u + 2 * e[..., None] + 22 * f32 * far[..., None] + 1e-5) * spread + 22 * f32 * farv
                 + 2.0 ** -25)
        err = np.abs(out - want)
        assert np.all(err <= bound), ((err - bound).max(), np.argwhere(~(err <= bound))[:4])
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(lse), none) and not out[none].any()
        le = np.abs(lse[~none] - want_lse[~none])
        limit = (e + 22 * f32 * far)[~none] + 1e-5 * (1 + np.abs(want_lse[~none]))
        assert np.all(le <= limit), (le - limit).max()


def extras(p, what, seed=0):
    """The named ones of softcap, slopes (of both signs), prefixes and documents for a problem."""
    import torch
    r = np.random.default_rng(seed)
    dev = lambda v, t: torch.tensor(np.asarray(v), dtype=t, device="cuda")  # noqa: E731
    kw = {}
    if "cap" in what:
        kw["softcap"] = 2.5
    if "slopes" in what:
        kw["slopes"] = dev([(0.5 if h % 3 else -0.01) * 2.0 ** (-h % 7) for h in range(p.heads)], torch.float32)
    if "prefix" in what:
        kw["prefix_lens"] = dev([r.integers(-2, max(2, int(kv * 1.2))) for _, kv in p.lens], torch.int32)
    if "docs" in what:
        starts = []
        for n, kv in p.lens:
            pos = np.arange(kv - n, kv)
            cuts = np.sort(r.integers(-5, max(1, kv), 6))
            starts += list(np.maximum.accumulate([max([c for c in cuts if c <= x], default=-3) for x in pos])) if n else []
        kw["doc_starts"] = dev(starts, torch.int32)
    return kw


SETS = ["cap", "slopes", "prefix", "docs", "cap slopes", "prefix docs", "cap slopes prefix docs"]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("what", SETS)
@pytest.mark.parametrize("heads,kv_heads,d,page,layout", [
    (4, 4, 128, 16, "slots_first"), (8, 2, 64, 32, "heads_first"), (15, 3, 72, 64, "one_buffer"), (16, 1, 128, 1024, "slots_first"),
])
def test_single_tokens(heads, kv_heads, d, page, layout, what, dtype):
    p = Scored([(1, n) for n in (1, 16, 0, 17, 63, 64, 65, 129, 700, 0, 1311)], heads, kv_heads, d, page, dtype, layout,
               seed=heads)
    kw = extras(p, what, heads)
    got = p.verify(**kw)
    again = kaio.paged_attention(p.q, p.kc, p.vc, p.table, p.kv, return_lse=True, **kw)
    assert all((a == b).all() for a, b in zip(got, again))
    p.verify(window=40, sinks=5, **kw)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("what", SETS)
@pytest.mark.parametrize("heads,kv_heads,d,page,lens", [
    (4, 4, 128, 16, [(130, 130)]),
    (8, 2, 128, 16, [(5, 300), (0, 77), (64, 64), (1, 500), (33, 129)]),
    (5, 1, 80, 64, [(100, 333), (2, 2), (40, 41)]),
    (2, 2, 16, 32, [(300, 300), (0, 0), (127, 128)]),
])
def test_chunks(heads, kv_heads, d, page, lens, what, dtype):
    p = Scored(lens, heads, kv_heads, d, page, dtype, seed=d)
    kw = extras(p, what, d)
    p.verify(**kw)
    if dtype == "float16":
        p.verify(window=50, sinks=3, **kw)


@pytest.mark.parametrize("what", ["cap slopes prefix docs", "prefix docs"])
@pytest.mark.parametrize("lens", [[(200, 700)], [(3, 70), (2, 30)]])
def test_not_causal(lens, what):
    p = Scored(lens, 4, 1, 64, 16, seed=3)
    p.verify(causal=False, **extras(p, what, 1))
    p.verify(causal=False, window=30, sinks=2, **extras(p, what, 2))


@pytest.mark.parametrize("lens", [[(4, 0)], [(5, 2)], [(200, 100), (1, 1)], [(300, 7), (2, 200)]])
def test_more_new_tokens_than_positions(lens):
    p = Scored(lens, 4, 2, 64, 16, seed=4)
    for what in SETS:
        p.verify(**extras(p, what, 5))


@pytest.mark.parametrize("n", [1, 2, 90])
def test_documents_that_hide_everything(n):
    """Rows without a visible key between rows with some; a begin behind the token's own place."""
    import torch
    p = Scored([(n, 200), (n, 150)], 4, 2, 128, 16, seed=6)
    for ds in (500, 2 ** 31 - 1, 201, 200 - n):
        docs = torch.tensor([-7] * (n - n // 2) + [ds] * (n // 2 + n), dtype=torch.int32, device="cuda")
        for kw in ({}, dict(window=20, sinks=4), dict(softcap=2.0), dict(prefix_lens=torch.tensor([60, 0], dtype=torch.int32, device="cuda"))):
            p.verify(doc_starts=docs, **kw)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("softcap,spread,scale", [(0.05, 3.0, None), (30.0, 60.0, None), (256.0, 1.0, None),
                                                  (5.0, 8.0, -0.3), (20.0, 1.0, 0.0), (1.0, 200.0, 4.0)])
def test_caps_small_large_and_far_exceeded(softcap, spread, scale, n):
    """Scores of hundreds of caps, negative and zero scales."""
    for dtype in ("float16", "bfloat16"):
        p = Scored([(n, 300), (n, 64)], 4, 2, 128, 16, dtype, seed=8, spread=spread)
        kw = dict(softcap=softcap) | ({} if scale is None else dict(scale=scale))
        p.verify(**kw)
        p.verify(**kw, **extras(p, "slopes docs", 3))


@pytest.mark.parametrize("n", [1, 70])
def test_slopes_far_and_steep(n):
    import torch
    p = Scored([(n, 5000)], 4, 4, 64, 64, seed=9)
    for s in ([0.0, 1.0, 100.0, 2.0 ** -8], [-2.0 ** -6, -0.5, 1e-30, 3.0]):
        p.verify(slopes=torch.tensor(s, device="cuda"))


@pytest.mark.parametrize("n", [1, 40])
def test_what_is_hidden_may_hold_anything(n):
    """NaN and infinities in k and v where nothing looks: before the first document, behind the
    end, between sink tokens and window; and in k alone where some rows look."""
    import torch
    p = Scored([(n, 300)], 4, 2, 64, 16, seed=10)
    ids = p.table[0].long()

    def fill(lo, hi, k, v):
        for j in range(lo, hi):
            if k is not None:
                p.kc[ids[j // 16], j % 16] = k
            if v is not None:
                p.vc[ids[j // 16], j % 16] = v

    docs = torch.full((n,), 100, dtype=torch.int32, device="cuda")
    kws = [dict(doc_starts=docs), dict(doc_starts=docs, softcap=2.0, slopes=torch.full((4,), 0.1, device="cuda"))]
    refs = [p.ref(**kw) for kw in kws]
    fars = [dict(p.far)] * 2
    for bad in (float("nan"), float("inf"), -float("inf")):
        fill(0, 100, bad, bad)
        fill(300, len(ids) * 16, bad, bad)
        for kw, ref, far in zip(kws, refs, fars):
            p.far, p.cap = far, kw.get("softcap", 0.0)
            p.check(p.run(**kw), ref)


def test_scored_results_belong_to_the_given_stream_and_replay():
    """Captured into a graph and replayed on new lengths, documents and inputs."""
    import torch
    for n in (1, 50):
        p = Scored([(n, 200), (n, 333)], 4, 2, 64, 16, seed=11)
        kw = extras(p, "cap slopes prefix docs", 4)
        ws = kaio.paged_attention_workspace()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        p.run(workspace=ws, stream=s, **kw)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = p.run(workspace=ws, **kw)
        for seed in (1, 2):
            q = Scored([(n, 150 + seed), (n, 240)], 4, 2, 64, 16, seed=20 + seed)
            for to, new in ((p.q, q.q), (p.kc, q.kc), (p.vc, q.vc)):
                to.copy_(new[:to.shape[0]] if new.shape[0] >= to.shape[0] else torch.cat((new, to[new.shape[0]:])))
            p.lens = q.lens
            p.kv.copy_(q.kv)
            p.table[:, :q.table.shape[1]].copy_(q.table)
            new = extras(p, "cap slopes prefix docs", seed)
            for k in ("slopes", "prefix_lens", "doc_starts"):
                kw[k].copy_(new[k])
            graph.replay()
            p.check(got, p.ref(**kw))
    kaio.device_status()


def test_without_extras_the_result_is_the_plain_one():
    import torch
    for n in (1, 60):
        p = Scored([(n, 300)], 4, 2, 128, 16, seed=12)
        a = p.run()
        b = p.run(softcap=0.0, doc_starts=torch.zeros(n, dtype=torch.int32, device="cuda"))
        c = p.run(slopes=torch.zeros(4, device="cuda"), prefix_lens=torch.zeros(1, dtype=torch.int32, device="cuda"))
        p.check(b, p.ref())
        p.check(c, p.ref())
        assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


def test_many_tiles_in_documents():
    """More row tiles than the sum over a sequence's items takes at a time; parts of items joined."""
    p = Scored([(700, 900), (1, 2000), (300, 300)], 8, 1, 64, 16, "bfloat16", seed=13)
    p.verify(**extras(p, "cap slopes prefix docs", 9))
    p.verify(**extras(p, "docs", 10))


@pytest.mark.parametrize("n", [1, 60])
def test_rows_behind_the_last_sequence_stay(n):
    """A padded batch: more rows of q, documents and results than the sequences have tokens."""
    import torch
    p = Scored([(n, 200), (n, 90)], 4, 2, 64, 16, seed=14)
    kw = extras(p, "cap slopes prefix docs", 6)
    want = p.run(**kw)
    pad = lambda t, v: torch.cat((t, torch.full((5, *t.shape[1:]), v, dtype=t.dtype, device="cuda")))  # noqa: E731
    out, lse = torch.full((2 * n + 5, 4, 64), 7.0, device="cuda").half(), torch.full((2 * n + 5, 4), 7.0, device="cuda")
    wide = dict(kw, doc_starts=pad(kw["doc_starts"], -1))
    p.run(q=pad(p.q, float("nan")), out=out, lse=lse, **wide)
    assert (out[:2 * n] == want[0]).all() and (lse[:2 * n] == want[1]).all()
    assert (out[2 * n:] == 7).all() and (lse[2 * n:] == 7).all()


def test_two_calls_at_once_on_streams_of_their_own():
    import torch
    a, b = Scored([(70, 900)], 8, 2, 64, 16, seed=15), Scored([(1, 3000), (1, 40)], 8, 2, 64, 16, seed=16)
    kws = [extras(p, "cap slopes docs", 7) for p in (a, b)]
    want = [p.run(**kw) for p, kw in zip((a, b), kws)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [kaio.paged_attention_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [p.run(workspace=ws, stream=s, **kw) for p, kw, ws, s in zip((a, b), kws, spaces, streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all((i == j).all() for i, j in zip(x, y))
