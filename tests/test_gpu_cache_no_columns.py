"""Forks of books whose table has no columns: only the lengths follow the parents."""
import random

import pytest

from test_gpu_cache import Books, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [2, 512, 513, 700, 8192])
def test_forks_without_columns(batch):
    b = Books(batch, 0, 0, 16, seed=batch)
    b.lens[:] = [i % 50 for i in range(batch)]
    b.d_lens.copy_(dev(b.lens))
    r = random.Random(batch)
    b.fork([r.randint(-1, batch) for _ in range(batch)])
    b.truncate([r.randint(-1, 60) for _ in range(batch)])
