"""Slopes near the largest number, whose biases pass f32's range (tolerance: that of test_gpu_paged_scored.py)."""
import pytest

from test_gpu_paged_scored import Scored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [0.0, 2.5])
@pytest.mark.parametrize("lens", [[(1, 1), (1, 400)], [(70, 197), (1, 300)], [(200, 200)]])
def test_slopes_near_the_largest_number(lens, softcap):
    """Biases past f32's range: only the token's own key is left."""
    import torch
    p = Scored(lens, 4, 4, 64, 16, seed=31)
    for slopes in ([3.4e38, 2.4e38, 2.3e38, 1e38], [1e37, 2e36, 1e36, 1e35]):
        p.verify(slopes=torch.tensor(slopes, device="cuda"), softcap=softcap)
