"""The distance bias where it is steep: nearly all weight lies on the nearest keys, whose own
biases are small or zero.

Tolerance: that of test_gpu_paged_scored.py. Its 22 * 2^-24 of a key's own bias holds for the chunks'
tiles left of a row, too: slope * log2(e) is rounded once, the product of it and the distance to the
nearest key of 32 once, and each of up to seven additions on the way out to a key is off by at
most 2^-24 of a partial sum that is no larger than the key's bias: nine, and one for the sum with the score.
"""
import pytest

from test_gpu_paged_scored import Scored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("softcap", [0.0, 2.5])
@pytest.mark.parametrize("lens,heads,kv_heads,d", [
    ([(70, 197)], 4, 4, 64), ([(130, 257), (33, 160)], 4, 4, 128), ([(40, 167)], 4, 2, 64), ([(300, 1323)], 4, 1, 64),
    ([(3, 130), (1, 128)], 4, 4, 64),
])
def test_steep_slopes_at_every_place_of_a_tile(lens, heads, kv_heads, d, softcap, dtype):
    """Warps whose first row is the last key of a tile, or just behind it."""
    import torch
    p = Scored(lens, heads, kv_heads, d, 16, dtype, seed=heads + d)
    for slopes in ([0.9, 50.0, 100.0, 1000.0], [1e5, 0.3, -0.01, 3e7]):
        p.verify(slopes=torch.tensor(slopes, device="cuda"), softcap=softcap)
