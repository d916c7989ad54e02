"""What no token sees may hold anything: NaN and infinities in k and v between the leading
positions (sinks, prefix) and the window, before the first document and behind the end, inside a tile
and across tiles; and in k alone at keys that some tokens see, which the others do not notice.

Tolerance: that of test_gpu_paged_scored.py, against the definition over clean memory.
"""
import numpy as np
import pytest

from oracle.attention import visible
from test_gpu_paged_scored import Scored

pytestmark = pytest.mark.gpu
BAD = (float("nan"), float("inf"), -float("inf"))

# (new, positions, window, sinks, prefix, documents' begins of the first and the second half)
PLACES = [
    (1, 700, 100, 10, 0, (0, 0)), (1, 700, 100, 3, 70, (33, 33)), (1, 190, 100, 70, 0, (65, 65)), (2, 700, 300, 0, 40, (20, 30)),
    (4, 260, 60, 0, 0, (100, 257)), (40, 700, 100, 10, 0, (0, 0)), (40, 700, 260, 3, 70, (33, 33)), (40, 239, 100, 70, 0, (9, 66)),
    (90, 900, 128, 5, 200, (130, 850)), (130, 640, 255, 129, 64, (127, 200)), (300, 1000, 50, 1, 0, (0, 5)), (60, 400, 0, 0, 0, (150, 365)),
    (200, 700, 0, 0, 300, (128, 128)),
]


def fill(p, where, k, v):
    import torch
    j = torch.as_tensor(np.flatnonzero(where), device="cuda")
    ids = p.table[0].long()[j // p.page]
    if k is not None:
        p.kc[ids, j % p.page] = k
    if v is not None:
        p.vc[ids, j % p.page] = v


def keywords(case, what):
    import torch
    n, kv, window, sinks, prefix, (d0, d1) = case
    dev = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    kw = dict(window=window, sinks=sinks, prefix_lens=dev([prefix]), doc_starts=dev([d0] * (n // 2) + [d1] * (n - n // 2)))
    if "cap" in what:
        kw["softcap"] = 2.0
    if "slopes" in what:
        kw["slopes"] = dev([0.3, 0.02, 0.0, -0.003], torch.float32)
    return kw


def seen_by(case):
    n, kv, window, sinks, prefix, (d0, d1) = case
    return visible(n, kv, True, window, sinks, prefix, [d0] * (n // 2) + [d1] * (n - n // 2))


@pytest.mark.parametrize("what", ["", "cap", "slopes", "cap slopes"])
@pytest.mark.parametrize("case", PLACES)
def test_memory_that_no_token_sees(case, what):
    n, kv = case[:2]
    for dtype, d in (("float16", 64), ("bfloat16", 128)):
        p = Scored([(n, kv)], 4, 2, d, 16, dtype, seed=51)
        kw = keywords(case, what)
        ref, far = p.ref(**kw), p.far
        hidden = np.ones(16 * p.table.shape[1], dtype=bool)
        hidden[:kv] = ~seen_by(case).any(0)
        for bad in BAD:
            fill(p, hidden, bad, bad)
            p.far, p.cap = far, kw.get("softcap", 0.0)
            p.check(p.run(**kw), ref)


@pytest.mark.parametrize("what", ["", "cap", "slopes", "cap slopes"])
@pytest.mark.parametrize("case", [c for c in PLACES if c[0] > 1])
def test_keys_that_only_some_tokens_see(case, what):
    n, kv = case[:2]
    p = Scored([(n, kv)], 4, 2, 64, 16, seed=52)
    kw = keywords(case, what)
    seen = seen_by(case)
    some = seen.any(0) & ~seen.all(0)
    for j in np.flatnonzero(some)[[0, -1]]:
        clean = p.kc.clone()
        ref, far = p.ref(**kw), p.far
        only = np.arange(kv) == j
        rows = ~seen[:, j]
        fill(p, only, float("nan"), None)
        out, lse = p.run(**kw)
        assert out[~rows].isnan().all() and lse[~rows].isnan().all()
        keep = lambda x: x[rows]  # noqa: E731
        p.far, p.cap = {k: keep(v) for k, v in far.items()}, kw.get("softcap", 0.0)
        p.check((keep(out), keep(lse)), tuple(keep(x) for x in ref))
        p.kc.copy_(clean)
