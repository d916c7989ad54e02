"""Capped scores of keys that hold infinities where tokens see them: the cap of an infinite score is
the cap itself, with its sign.

Tolerance: that of test_gpu_paged_scored.py with S taken of the keys as they were (an infinite
score has no error but the cap's own).
"""
import pytest

from test_gpu_paged_scored import Scored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [2.5, 30.0, 256.0])
@pytest.mark.parametrize("n,kv", [(1, 300), (40, 300), (200, 200), (90, 900)])
def test_infinite_scores_are_caps(n, kv, softcap):
    import torch
    for sign in (-1.0, 1.0):
        for lo, hi in ((0, 128), (0, kv), (5, 6), (100, 290)):
            p = Scored([(n, kv)], 4, 2, 64, 16, seed=41)
            p.q[..., 0] = 1.0
            for kw in (dict(softcap=softcap), dict(softcap=softcap, slopes=torch.full((4,), 0.02, device="cuda"))):
                size = p.ref(**kw)[3]
                ids = p.table[0].long()
                for j in range(lo, min(hi, kv)):
                    p.kc[ids[j // 16], j % 16, :, 0] = sign * float("inf")
                want, lse, spread, _ = p.ref(**kw)
                p.check(p.run(**kw), (want, lse, spread, size))
