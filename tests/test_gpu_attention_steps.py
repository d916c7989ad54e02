"""The projections, the rotation with its cache write and the attention run together, as
the example does, against the oracles chained in 64 bits.

Tolerance: the projections' f16 results are compared by their own tests; here they are
taken from the kernel, so that what follows starts from the same values. k is rounded to
f16 in the cache (2^-11 of each value), and so is the rotated q: each score is then off
by at most 2 * 2^-11 * S (S = |scale| max_j sum_d |q_d k_jd|) beside the attention's own
error, a weight by that much relative, and the output by twice that times A = sum_j p_j
|v_j|.
"""
import os
import sys

import numpy as np
import pytest

from oracle.attention import paged_attention_ref, rope_ref
from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_chunks_then_tokens(window, sinks):
    import torch
    from attention_steps import PagedLayer
    columns, heads, d = 256, 3, 64
    layer = PagedLayer(columns, heads, d, 3, pages=40, window=window, sinks=sinks, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    inv = layer.inv_freq.double().cpu().numpy()
    k_all, v_all = [[[] for _ in range(3)] for _ in range(2)]
    for new in ([37, 5, 60], [0, 20, 1], [1, 1, 1], [1, 1, 1], [9, 1, 0]):
        x = torch.randn(sum(new), columns, generator=g, device="cuda").half()
        first = list(layer.lengths)
        out = layer.step(x, new).double().cpu().numpy().reshape(-1, heads, d)
        q, k, v = (t.double().cpu().numpy().reshape(-1, heads, d)
                   for t in kaio.qkv_project_int4(x, *layer.weights, *layer.scales))
        row = 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            pos = np.arange(first[b], first[b] + n)[None]
            k_all[b].append(rope_ref(k[row:row + n], pos, inv, (d // 2,)))
            v_all[b].append(v[row:row + n])
            keys, values = np.concatenate(k_all[b])[None], np.concatenate(v_all[b])[None]
            want, _, spread, size = paged_attention_ref(rope_ref(q[row:row + n], pos, inv, (d // 2,)), keys, values,
                                                        [[0]], [keys.shape[1]], [0, n], d ** -0.5,
                                                        window=window, sinks=sinks)
            u = 2.0 ** -11
            bound = u * np.abs(want) + (u + 2 * (2 * u + (d + 8) * 2.0 ** -24) * (size[..., None] + 1) + 1e-5) * spread
            err = np.abs(out[row:row + n] - want)
            assert np.all(err <= bound + 2.0 ** -25), (err - bound).max()
            row += n
    kaio.device_status()


def test_the_example_runs():
    import attention_steps
    attention_steps.main()
