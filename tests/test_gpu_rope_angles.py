"""Rotary angles of frequencies above one, against angles reduced in 60 decimal digits.

The tolerance is that of test_gpu_rope.py: an angle within 2^-24 turns (3.8e-7 radians),
f32 sine, products and sum, together 1.01e-6 (|x0| + |x1|), and one rounding to f16."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.283185307179586476925286766559005768394338798750211641949889184615632812572418")


def reduced(position, frequency):
    """position * frequency modulo 2 pi, as a float; frequency a float32."""
    getcontext().prec = 60
    turns = Decimal(int(position)) * Decimal(float(frequency)) / TWO_PI
    return float((turns - turns.to_integral_value()) * TWO_PI)


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_above_one(interleaved):
    import torch
    freq = np.float32([1.0, 1.0000001, 1.5, 8.0, 8.1, 64.3, 1000.0, 1234.567, 65536.1, 3.3e6, 1e9, 2.0 ** 40 * 1.7, 2.0 ** 63 * 1.1, -8.1,
                       -1000.0, 0.0, 1e-30, -1e-30, 0.3])
    pos = np.int32([0, 1, -1, 3, 100003, 16777217, 2**30 + 12345, 2**31 - 1, -2**31])
    t, r = len(pos), len(freq)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(t, 2, 2 * r + 2, device="cuda", generator=g).half()
    got = kaio.rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), interleaved=interleaved)
    angle = np.array([[reduced(p, f) for f in freq] for p in pos])[:, None, :]
    x64, out = (v.double().cpu().numpy() for v in (x, got))
    i = np.arange(r)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    x0, x1 = x64[..., a], x64[..., b]
    size = np.abs(x0) + np.abs(x1)
    for at, want in ((a, x0 * np.cos(angle) - x1 * np.sin(angle)), (b, x1 * np.cos(angle) + x0 * np.sin(angle))):
        err, bound = np.abs(out[..., at] - want), 2.0 ** -11 * np.abs(want) + 1.01e-6 * size + 2.0 ** -25
        assert np.all(err <= bound), [(float(freq[c]), int(pos[p]), float(e)) for p, h, c in np.argwhere(err > bound)[:9]
                                      for e in [err[p, h, c]]]
