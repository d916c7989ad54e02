"""The cache's upkeep together with the projections, the rotation and the attention, as the
example uses them: prompts, forks, drafts that are cut, sequences that end, a compaction, and
the attention's results against the oracle over what each sequence should hold.

Tolerance: as in test_gpu_attention_steps.py (k and q rounded to f16 after the rotation), with
24 * 2^-24 caps more for each score where they are capped, and 22 * 2^-24 of the bias where
there are slopes.
"""
import os
import sys

import numpy as np
import pytest

from oracle import cache
from oracle.attention import paged_attention_ref, rope_ref
from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("softcap,slopes,window,sinks", [(0.0, None, 0, 0), (1.5, None, 0, 0), (0.0, [0.25, 0.03], 0, 0),
                                                         (2.0, [0.1, 0.0], 24, 5)])
def test_forked_drafted_cut_and_compacted(softcap, slopes, window, sinks):
    import torch
    from attention_steps import PagedLayer
    columns, heads, d, rows = 256, 2, 64, 4
    slopes = None if slopes is None else torch.tensor(slopes, device="cuda")
    layer = PagedLayer(columns, heads, d, rows, pages=60, window=window, sinks=sinks, seed=3, softcap=softcap, slopes=slopes)
    g = torch.Generator(device="cuda").manual_seed(4)
    inv = layer.inv_freq.double().cpu().numpy()
    held = [([], []) for _ in range(rows)]                 # rotated k and v of every position of each row

    def step(new):
        x = torch.randn(sum(new), columns, generator=g, device="cuda").half()
        first = list(layer.lengths)
        out = layer.step(x, new).double().cpu().numpy().reshape(-1, heads, d)
        q, k, v = (t.double().cpu().numpy().reshape(-1, heads, d)
                   for t in kaio.qkv_project_int4(x, *layer.weights, *layer.scales))
        at = 0
        for b, n in enumerate(new):
            if n:
                pos, part = np.arange(first[b], first[b] + n)[None], slice(at, at + n)
                held[b][0].extend(rope_ref(k[part], pos, inv, (d // 2,)))
                held[b][1].extend(v[part])
                far = {}
                want, _, spread, size = paged_attention_ref(
                    rope_ref(q[part], pos, inv, (d // 2,)), np.stack(held[b][0])[None], np.stack(held[b][1])[None], [[0]],
                    [len(held[b][0])], [0, n], d ** -0.5, window=window, sinks=sinks, softcap=softcap,
                    slopes=None if slopes is None else slopes.tolist(), far=far)
                u, f32 = 2.0 ** -11, 2.0 ** -24
                e = (2 * u + (d + 8) * f32) * (size[..., None] + 1) + 24 * f32 * softcap
                bias = 22 * f32 * (far["b"][..., None] * spread + far["bv"]) if far else 0.0
                bound = u * np.abs(want) + (u + 2 * e + 1e-5) * spread + bias
                err = np.abs(out[part] - want)
                assert np.all(err <= bound + 2.0 ** -25), (b, (err - bound).max())
            at += n
        check()

    def check():
        refs, table, lens = (t.tolist() for t in layer.books())
        assert lens == layer.lengths == [len(k) for k, _ in held]
        assert refs == cache.count(table, lens, layer.page_size, len(refs))

    step([37, 5, 60, 16])
    step([1, 1, 1, 1])
    layer.fork([2, 1, 2, 2])
    held = [(list(held[b][0]), list(held[b][1])) for b in (2, 1, 2, 2)]
    check()
    step([1, 0, 1, 1])                                     # each fork's last page becomes its own
    step([6, 3, 1, 20])
    cut = [layer.lengths[0] - 5, 0, 10 ** 9, layer.lengths[3] - 17]
    layer.truncate(cut)
    held = [(k[:n], v[:n]) for (k, v), n in zip(held, cut)]
    check()
    layer.fork([3, 0, 2, 0])
    held = [(list(held[b][0]), list(held[b][1])) for b in (3, 0, 2, 0)]
    layer.compact()
    check()
    used = int((layer.page_refs > 0).sum())
    assert bool((layer.page_refs[:used] > 0).all())
    step([2, 40, 1, 1])
    step([1, 1, 1, 1])
    layer.truncate([0] * rows)
    held = [([], []) for _ in range(rows)]
    check()
    assert not layer.page_refs.any()
    kaio.device_status()
