"""Attention where many keys far below one make up the result: a few keys (the first
tokens, say) take nearly all the weight and have values of zero.

Tolerance: that of test_gpu_paged_attention.py, whose u * A bounds the weights' rounding
as long as they are normal numbers of their type. f16 weights are held relative to a
reference that makes the largest of them at least 2^7, so what lies below 2^-21 of it is
an f16 subnormal, off by up to 2^-25 of 2^7: for every key another 2^-32 |v|.
"""
import numpy as np
import pytest

from oracle.attention import paged_attention_ref
from test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu


def problem(lens, bits, dtype, d=64, heads=4, kv_heads=2):
    """Every 16th of the first 64 positions scores `bits` (in log2) above all others."""
    import torch
    p = Problem(lens, heads, kv_heads, d, 16, dtype, seed=int(bits))
    p.scale = 0.125
    p.q.zero_()
    p.q[..., 0] = 8.0
    p.kc.zero_()
    p.vc.copy_((1.0 + 0.1 * p.vc.float().clamp(-3, 3)) * 2.0 ** min(bits - 8, 14))
    for b, (_, kv) in enumerate(lens):
        for j in range(0, min(kv, 64), 16):
            at = (int(p.table[b, j // 16]), j % 16)
            p.kc[at][:, 0] = bits * float(np.log(2.0))
            p.vc[at].zero_()
    assert torch.isfinite(p.vc).all()
    return p


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits", [10.3, 18.3, 22.3, 25.6])
@pytest.mark.parametrize("lens,mask", [
    ([(1, 512)], {}), ([(1, 512), (1, 9000), (1, 300)], {}), ([(2, 4000)], dict(window=3000, sinks=64)),
    ([(100, 700)], {}), ([(200, 2500), (1, 1500), (20, 900)], {}), ([(150, 1500)], dict(window=1000, sinks=64)),
])
def test_small_weights_add_up(lens, mask, bits, dtype):
    p = problem(lens, bits, dtype)
    got = p.run(scale=p.scale, **mask)
    out, lse, spread, size = p.ref(**mask)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    every = paged_attention_ref(f(p.q) * 0, f(p.kc), np.abs(f(p.vc)), p.table.cpu().numpy(), p.kv.tolist(),
                                p.starts.tolist(), 1.0, True, mask.get("window", 0), mask.get("sinks", 0))
    keys = np.exp(every[1])                     # with scores of zero: how many a token sees
    u = 2.0 ** {"float16": -11, "bfloat16": -8}[dtype]
    e = (p.d + 8) * 2.0 ** -24 * (size + 1)
    lost = 2.0 ** -32 * keys[..., None] * every[0] if dtype == "float16" else 0.0
    bound = u * np.abs(out) + (u + 2 * e[..., None] + 1e-5) * spread + 2.0 ** -25 + lost
    err = np.abs(f(got[0]) - out)
    assert np.all(err <= bound), (err / bound).max()
    assert np.all(np.abs(f(got[1]) - lse) <= e + 1e-5 * (1 + np.abs(lse)))


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("log2_scale", range(0, 6))
def test_large_scores_keep_weights_in_range(n, log2_scale):
    """Scores of 2^22 and more, whose f32 steps come to the size of the exponents' shift, and
    which rise late by one step: a result is still a mean of values, weighted by numbers
    that are rounded once (2^-11 each), and lse the largest score but for ln(keys) and
    three roundings of that score."""
    import torch
    scale = 2.0 ** log2_scale
    p = Problem([(n, 400)], 2, 1, 64)
    p.q.zero_()
    p.kc.zero_()
    p.q[..., 0], p.q[..., 1] = 2048.0, 1.0
    p.kc[..., 0] = 2048.0
    for j in range(384, 400):
        p.kc[p.table[0, j // 16], j % 16, :, 1] = 1.0
    out, lse = p.run(scale=scale, causal=False)
    assert (out.double().abs() <= float(p.vc.abs().max()) * (1 + 2.0 ** -10)).all()
    top = scale * (2.0 ** 22 + 1)
    assert ((lse.double() - top).abs() <= np.log(400) + 3 * 2.0 ** -24 * top).all()
