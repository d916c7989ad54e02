"""Pools and tables past the sizes at which a cluster of 16 CTAs looks after them, and past those
at which a warp keeps more than 32 words of pages."""
import random

import pytest

from oracle import cache
from test_gpu_cache import Books, dev

pytestmark = pytest.mark.gpu


def scattered(batch, width, pages, page, seed):
    """Rows that hold pages from all over the pool, with gaps between them."""
    b = Books(batch, width, pages, page, seed=seed)
    r = random.Random(seed)
    held = r.sample(range(pages), batch * (width - 2))
    for row in range(batch):
        ids = held[row * (width - 2):(row + 1) * (width - 2)]
        b.table[row][:len(ids)] = ids
        b.lens[row] = page * len(ids) - (row % page)
    b.refs[:] = cache.count(b.table, b.lens, page, pages)
    b.d_table.copy_(dev(b.table)), b.d_lens.copy_(dev(b.lens)), b.d_refs.copy_(dev(b.refs))
    return b


@pytest.mark.parametrize("batch,width,pages", [(8, 8000, 140001), (5, 3000, 300000), (4, 40000, 524289), (3, 100000, 1100000)])
def test_sixteen_ctas(batch, width, pages):
    b = scattered(batch, width, pages, 4, pages)
    b.compact(4096)
    b.append([7, 0, 1][:batch] + [4] * (batch - 3))
    b.fork([1, 0, 1][:batch] + [2] * (batch - 3))
    b.append([1] * batch)
    b.truncate([n - 4 * (width // 3) for n in b.lens])
    b.compact(pages)
    used = sum(x > 0 for x in b.refs)
    assert all(x > 0 for x in b.refs[:used])


@pytest.mark.parametrize("pages", [524289, 1100000])
def test_free_pages_at_the_pool_s_end_alone(pages):
    """All lower pages are held, so what is free lies in the last words of the last warps."""
    b = Books(2, pages // 2, pages, 2, seed=3)
    first = pages // 2 - 3
    b.table[0][:first], b.table[1][:first] = range(first), range(first, 2 * first)
    b.lens[:] = [2 * first, 2 * first - 1]
    b.refs[:] = cache.count(b.table, b.lens, 2, pages)
    b.d_table.copy_(dev(b.table)), b.d_lens.copy_(dev(b.lens)), b.d_refs.copy_(dev(b.refs))
    b.append([2, 4])
    b.truncate([9, 2 * first])
    b.append([5, 1])
    b.compact(100)
