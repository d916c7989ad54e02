"""The cache's upkeep where a device places fewer thread blocks as one cluster than would be taken."""
import random

import pytest

from qkv_projection_gb300 import kaio
from test_gpu_cache import Books, dev
from test_gpu_cache_large_pools import scattered

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2, 3, 8, 12, 16])
def most(request, monkeypatch):
    """The calls of kaio go through the entry with a limit."""
    L, limit = kaio.lib(), request.param

    class Limited:
        def __getattr__(self, name):
            ops = ("kaio_cache_fork", "kaio_cache_append", "kaio_cache_compact")
            if name not in ops:
                return getattr(L, name)
            return lambda args, stream: L.kaio_debug_cache_cluster_limit(ops.index(name), args, limit, stream)

    monkeypatch.setattr(kaio, "_host", lambda: False)
    monkeypatch.setattr(kaio, "_host_module", False)
    monkeypatch.setattr(kaio, "lib", lambda: Limited())
    return limit


def test_steps_within_the_limit(most):
    r = random.Random(most)
    b = Books(33, 30, 1500, 16, stride=37, seed=most)
    for _ in range(20):
        b.step(60)
    b = Books(40, 300, 40000, 4, seed=most)
    for _ in range(6):
        b.append([r.randint(0, 60) for _ in range(40)])
        b.fork([r.randrange(40) for _ in range(40)])
        b.truncate([r.randint(0, 200) for _ in range(40)])
        b.compact(50)


def test_large_pools_within_the_limit(most):
    b = scattered(8, 8000, 140001, 4, 5)
    b.compact(4096)
    b.append([7, 0, 1, 4, 4, 4, 4, 4])
    b.fork([1, 0, 1, 2, 2, 2, 2, 2])
    b.truncate([n // 2 for n in b.lens])
    b.compact(140001)


def test_pools_that_do_not_fit_are_refused(most):
    """2^23 pages and 8192 rows: 64 KB of words in each of 16 thread blocks, 128 in 8."""
    import torch
    rows, pages = 8192, 1 << 23
    books = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros(rows, 2, dtype=torch.int32, device="cuda"), dev([0] * rows)
    if most >= 12:
        slots, src, dst = kaio.cache_append(*books, None, rows, 16)
        assert slots.tolist() == [16 * i for i in range(rows)] and (src == -1).all() and (dst == -1).all()
        return
    with pytest.raises(kaio.KaioError, match="thread blocks"):
        kaio.cache_append(*books, None, rows, 16)
    assert not books[0].any() and not books[2].any()
    if most < 8:
        with pytest.raises(kaio.KaioError, match="thread blocks"):
            kaio.cache_compact(*books, 16, 3)
    else:
        books[0][5], books[1][7, 0], books[2][7] = 1, 5, 3
        src, dst = kaio.cache_compact(*books, 16, 3)
        assert src.tolist() == [5, -1, -1] and dst.tolist() == [0, -1, -1]
        assert int(books[1][7, 0]) == 0 and int(books[0][0]) == 1 and int(books[0].sum()) == 1


def test_a_first_call_under_capture():
    """What is asked once for a device may be asked while a graph is captured, in a thread of its own."""
    import threading

    import torch
    b = scattered(8, 8000, 140001, 4, 6)
    parents, starts = dev([1, 0, 1, 2, 2, 2, 2, 2]), dev([0, 7, 7, 8, 12, 16, 20, 24, 28])
    graph, made, errors = torch.cuda.CUDAGraph(), [], []

    def capture():
        try:
            with torch.cuda.graph(graph):
                kaio.cache_fork(*b.books(), parents, 4)
                made.extend(kaio.cache_append(*b.books(), starts, 28, 4))
                made.extend(kaio.cache_compact(*b.books(), 4, 100))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=capture)
    t.start()
    t.join()
    assert not errors, errors
    graph.replay()
    torch.cuda.synchronize()
    from oracle import cache
    cache.fork(b.refs, b.table, b.lens, parents.tolist(), 4)
    want = cache.append(b.refs, b.table, b.lens, starts.tolist(), 28, 4)
    want += cache.compact(b.refs, b.table, b.lens, 4, 100)
    assert [t.tolist() for t in made] == list(want)
    b.same()
