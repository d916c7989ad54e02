"""The cache's upkeep on the GPU against the books' oracle: whole numbers, equal everywhere,
the places that nobody holds included."""
import random

import pytest

from oracle import cache
from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu


def dev(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Books:
    """The oracle's lists and the GPU's arrays side by side."""

    def __init__(self, batch, width, pages, page, stride=0, seed=0):
        import torch
        self.r = random.Random(seed)
        self.batch, self.width, self.pages, self.page = batch, width, pages, page
        self.refs, self.lens = [0] * pages, [0] * batch
        self.table = [[self.r.randint(-9, pages + 9) for _ in range(width)] for _ in range(batch)]
        self.whole = torch.full((batch, max(stride, width)), 77, dtype=torch.int32, device="cuda")
        self.d_table = self.whole[:, :width]
        self.d_refs, self.d_lens = dev(self.refs), dev(self.lens)
        self.d_table.copy_(dev(self.table).reshape(batch, width))

    def books(self):
        return self.d_refs, self.d_table, self.d_lens

    def same(self):
        assert self.d_refs.tolist() == self.refs
        assert self.d_lens.tolist() == self.lens
        assert self.d_table.tolist() == self.table
        assert (self.whole[:, self.width:] == 77).all()

    def append(self, new, past=0, **kw):
        starts = [sum(new[:i]) for i in range(len(new) + 1)]
        tokens = starts[-1] + past
        got = kaio.cache_append(*self.books(), dev(starts), tokens, self.page, **kw)
        want = cache.append(self.refs, self.table, self.lens, starts, tokens, self.page)
        assert [g.tolist() for g in got] == list(want)
        self.same()
        return want

    def fork(self, parents):
        kaio.cache_fork(*self.books(), dev(parents), self.page)
        cache.fork(self.refs, self.table, self.lens, parents, self.page)
        self.same()

    def truncate(self, new):
        kaio.cache_truncate(*self.books(), dev(new), self.page)
        cache.truncate(self.refs, self.table, self.lens, new, self.page)
        self.same()

    def compact(self, moves):
        got = kaio.cache_compact(*self.books(), self.page, moves)
        want = cache.compact(self.refs, self.table, self.lens, self.page, moves)
        assert [g.tolist() for g in got] == list(want)
        self.same()
        return want

    def step(self, most):
        """Something at random."""
        r, b = self.r, self.batch
        what = r.choice(["append", "append", "fork", "truncate", "compact"])
        if what == "append":
            self.append([r.choice([0, 1, 1, r.randint(0, most)]) for _ in range(b)], past=r.choice([0, 3]))
        elif what == "fork":
            self.fork([r.choice([i, r.randrange(b), r.randint(-2, b + 1)]) for i in range(b)])
        elif what == "truncate":
            self.truncate([r.choice([2 ** 31 - 1, r.randint(-3, max(1, n)), n]) for n in self.lens])
        else:
            self.compact(r.choice([0, 1, 5, self.pages, 2 * self.pages]))


@pytest.mark.parametrize("seed", range(8))
def test_random_steps(seed):
    r = random.Random(100 + seed)
    page = r.choice([1, 3, 16, 48, 1024])
    batch = r.choice([1, 2, 5, 33])
    b = Books(batch, r.randint(1, 30), r.choice([1, 7, 40, 40 * batch]), page, stride=r.choice([0, 37]), seed=seed)
    for _ in range(25):
        b.step(5 * page)


@pytest.mark.parametrize("batch,width,pages,page", [
    (1, 3000, 4096, 16), (1500, 9, 20000, 16), (8192, 4, 30000, 1), (64, 250, 16 * 32 * 32 * 3, 16), (3, 5, 16 * 32 * 32 + 1, 4),
])
def test_large_books(batch, width, pages, page):
    b = Books(batch, width, pages, page, seed=batch)
    b.append([min(width * page, 1 + (i * 37) % (2 * page + 3)) for i in range(batch)])
    b.fork([(i * 7 + 1) % batch for i in range(batch)])
    b.append([1] * batch)
    b.truncate([n // 2 if i % 3 else 0 for i, n in enumerate(b.lens)])
    b.compact(100)
    b.compact(pages)
    used = sum(x > 0 for x in b.refs)
    assert all(x > 0 for x in b.refs[:used])
    b.append([b.r.randint(0, width * page) for _ in range(batch)])


def test_a_pool_that_runs_out():
    """Rows that do not fit take nothing; rows behind them that need no page go on."""
    b = Books(5, 4, 6, 4, seed=1)
    b.append([3, 16, 17, 2, 1])                       # 17 is past the row's places; six pages: 1 + 4 + 1, then none
    assert b.lens == [3, 16, 0, 2, 0]
    b.append([1, 0, 0, 3, 1])                         # row 0 fits its page, row 3 would need one
    assert b.lens == [4, 16, 0, 2, 0]
    b.fork([0, 0, 0, 3, 4])
    b.append([1, 1, 1, 2, 1])
    b.truncate([0] * 5)
    assert not any(b.refs)


def test_last_pages_that_are_shared():
    b = Books(4, 6, 30, 8, seed=2)
    b.append([13, 0, 0, 16])
    b.fork([0, 0, 0, 3])
    slots, src, dst = b.append([1, 2, 0, 1])
    assert src[0] == src[1] >= 0 and src[2:] == [-1, -1] and dst[0] != dst[1]
    assert b.refs[src[0]] == 1                        # the row that did not append keeps it
    slots, src, dst = b.append([1, 1, 1, 1])
    assert src == [-1] * 4


def test_one_token_each_by_default():
    b = Books(3, 4, 9, 2, seed=3)
    for _ in range(5):
        got = kaio.cache_append(*b.books(), None, 3, 2)
        want = cache.append(b.refs, b.table, b.lens, [0, 1, 2, 3], 3, 2)
        assert [g.tolist() for g in got] == list(want)
        b.same()


def test_nothing_at_all():
    import torch
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    none = (e, torch.empty(0, 0, dtype=torch.int32, device="cuda"), e)
    kaio.cache_fork(*none, e, 16)
    kaio.cache_truncate(*none, e, 16)
    assert all(t.numel() == 0 for t in kaio.cache_append(*none, None, 0, 16))
    assert all(t.numel() == 0 for t in kaio.cache_compact(*none, 16, 0))
    b = Books(2, 0, 0, 16)
    b.append([1, 0])
    b.fork([1, 0])
    b.truncate([0, 0])
    b.compact(3)


def test_lengths_and_entries_that_make_no_sense():
    """Lengths below zero and past the table, entries outside the pool: held as far as they go."""
    b = Books(4, 3, 10, 4, seed=5)
    b.lens[:] = [-3, 100, 5, 2 ** 31 - 1]
    b.table[1], b.table[2], b.table[3] = [2, -1, 99], [2 ** 31 - 1, 4, 0], [-2 ** 31 + 1, 10, 7]
    b.refs[:] = cache.count(b.table, b.lens, 4, 10)
    b.d_lens.copy_(dev(b.lens)), b.d_table.copy_(dev(b.table)), b.d_refs.copy_(dev(b.refs))
    b.append([1, 1, 1, 1])
    b.fork([3, 2, 1, 0])
    b.compact(10)
    b.truncate([1, 0, 2, 7])


@pytest.mark.parametrize("batch", [3, 700])
def test_forks_of_entries_of_every_value(batch):
    """A held entry outside the pool is copied as it stands, and what stood there before it is gone."""
    b = Books(batch, 12, 40, 4, seed=7)
    odd = (-2 ** 31, -2 ** 31 + 1, -1, 40, 2 ** 31 - 1)
    for i in range(batch):
        b.lens[i] = (13, 30, 0)[i % 3]
        b.table[i] = [odd[(i + j) % 5] if i % 3 else 7 for j in range(12)]
    b.d_lens.copy_(dev(b.lens))
    b.d_table.copy_(dev(b.table))
    b.refs[7] = 4 * len(b.lens[::3])
    b.d_refs.copy_(dev(b.refs))
    r = random.Random(batch)
    b.fork([1, 2, 1] + [r.randint(-1, batch) for _ in range(batch - 3)])
    b.fork([r.randint(-1, batch) for _ in range(batch)])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("layout", ["slots_first", "heads_first", "one_buffer", "padded", "sliced"])
@pytest.mark.parametrize("page,kv_heads,d,caches", [(16, 2, 64, 2), (1, 1, 8, 3), (32, 8, 128, 5), (24, 3, 72, 70), (1024, 1, 256, 1)])
def test_copied_pages(page, kv_heads, d, caches, layout, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(d)
    pages = 12
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(getattr(torch, dtype))  # noqa: E731
    full = {"slots_first": lambda: rnd(pages, page, kv_heads, d), "heads_first": lambda: rnd(pages, kv_heads, page, d),
            "one_buffer": lambda: rnd(pages, 2, page, kv_heads, d), "padded": lambda: rnd(pages, page, kv_heads, d + 16),
            "sliced": lambda: rnd(pages + 2, page + 3, kv_heads + 1, d)}[layout]
    view = {"slots_first": lambda t: t, "heads_first": lambda t: t.transpose(1, 2), "one_buffer": lambda t: t[:, 1],
            "padded": lambda t: t[..., 8:8 + d], "sliced": lambda t: t[1:-1, 2:page + 2, :kv_heads]}[layout]
    buffers = [full() for _ in range(caches)]
    want = [b.clone() for b in buffers]
    src, dst = [3, 0, -1, 3, 5, 12, 6, 2 ** 31 - 1], [1, 2, 4, 7, 12, 5, 6, 9]
    for w in want:
        for a, b in zip(src, dst):
            if 0 <= a < pages and 0 <= b < pages:
                view(w)[b] = view(w)[a].clone()
    kaio.cache_copy_pages([view(b) for b in buffers], dev(src), dev(dst))
    assert all(torch.equal(b, w) for b, w in zip(buffers, want))


def test_copies_of_unlike_layouts_together():
    import torch
    a = torch.randn(9, 16, 4, 64, device="cuda").half()
    b = torch.randn(9, 4, 16, 64, device="cuda").half()
    want = a.clone(), b.clone()
    want[0][7], want[1][7] = a[2], b[2]
    kaio.cache_copy_pages((a, b.transpose(1, 2)), dev([2]), dev([7]))
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    kaio.cache_copy_pages((a,), dev([]), dev([]))
    kaio.cache_copy_pages([], dev([1]), dev([2]))
    with pytest.raises(ValueError, match="caches.1."):
        kaio.cache_copy_pages((a, a[:, :8]), dev([2]), dev([7]))
    with pytest.raises(TypeError, match="float16 or"):
        kaio.cache_copy_pages((a.float(),), dev([2]), dev([7]))


def test_captured_steps_on_another_stream():
    """A fork, an append with its copies, a cut and a compaction as one graph, replayed."""
    import torch
    b = Books(6, 20, 150, 4, seed=8)
    b.append([9, 30, 2, 0, 17, 4])
    data = torch.randn(150, 4, 1, 8, device="cuda").half()
    starts, parents, kept = dev([0, 1, 3, 3, 8, 9, 10]), dev([1, 1, 0, 2, 5, 4]), dev([5, 31, 0, 4, 2, 20])
    start = [t.clone() for t in (*b.books(), data)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        kaio.cache_fork(*b.books(), parents, 4, stream=stream)
        slots, src, dst = kaio.cache_append(*b.books(), starts, 10, 4, stream=stream)
        kaio.cache_copy_pages([data], src, dst, stream=stream)
        kaio.cache_truncate(*b.books(), kept, 4, stream=stream)
        csrc, cdst = kaio.cache_compact(*b.books(), 4, 9, stream=stream)
        kaio.cache_copy_pages([data], csrc, cdst, stream=stream)
        return slots, src, dst, csrc, cdst

    first = step(s)
    s.synchronize()
    eager = [t.clone() for t in (*first, *b.books(), data)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    for _ in range(3):
        for to, new in zip((*b.books(), data), start):
            to.copy_(new)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip((*made, *b.books(), data), eager))
    cache.fork(b.refs, b.table, b.lens, parents.tolist(), 4)
    want = cache.append(b.refs, b.table, b.lens, starts.tolist(), 10, 4)
    cache.truncate(b.refs, b.table, b.lens, kept.tolist(), 4)
    want += cache.compact(b.refs, b.table, b.lens, 4, 9)
    assert [t.tolist() for t in made] == list(want)
    b.same()


def test_two_books_at_once_on_streams_of_their_own():
    """Kernels of one cluster and of one CTA side by side, many times."""
    import torch
    books = [Books(40, 300, 40000, 4, seed=21), Books(5, 30, 200, 4, seed=22)]
    streams = [torch.cuda.Stream() for _ in books]
    torch.cuda.synchronize()
    r = random.Random(5)
    results = [[] for _ in books]
    for _ in range(15):
        new = [[r.randint(0, 60 // (1 + k)) for _ in range(b.batch)] for k, b in enumerate(books)]
        kept = [[r.randint(0, 200) for _ in range(b.batch)] for b in books]
        parents = [[r.randrange(b.batch) for _ in range(b.batch)] for b in books]
        args = [[dev(v) for v in (([sum(n[:i]) for i in range(len(n) + 1)]), k, p)] for n, k, p in zip(new, kept, parents)]
        torch.cuda.synchronize()
        for k, (b, s, (starts, cut, par)) in enumerate(zip(books, streams, args)):
            got = kaio.cache_append(*b.books(), starts, sum(new[k]), 4, stream=s)
            kaio.cache_fork(*b.books(), par, 4, stream=s)
            kaio.cache_truncate(*b.books(), cut, 4, stream=s)
            got += kaio.cache_compact(*b.books(), 4, 50, stream=s)
            results[k].append((new[k], parents[k], kept[k], got))
    torch.cuda.synchronize()
    for b, steps in zip(books, results):
        for new, parents, kept, got in steps:
            starts = [sum(new[:i]) for i in range(len(new) + 1)]
            want = cache.append(b.refs, b.table, b.lens, starts, starts[-1], 4)
            cache.fork(b.refs, b.table, b.lens, parents, 4)
            cache.truncate(b.refs, b.table, b.lens, kept, 4)
            want += cache.compact(b.refs, b.table, b.lens, 4, 50)
            assert [g.tolist() for g in got] == list(want)
        b.same()


def test_results_of_a_call_that_ended_long_ago_are_its_own():
    """slots, src and dst of one call share memory with each other, and with no later call's."""
    b = Books(4, 8, 64, 4, seed=23)
    first = kaio.cache_append(*b.books(), dev([0, 3, 3, 9, 10]), 10, 4)
    kept = [t.clone() for t in first]
    for _ in range(5):
        kaio.cache_append(*b.books(), None, 4, 4)
        kaio.cache_compact(*b.books(), 4, 7)
    assert all((x == y).all() for x, y in zip(first, kept))
    assert first[0].is_contiguous() and first[0].shape == (10,) and first[1].shape == first[2].shape == (4,)
    first[0].zero_()
    assert (first[1] == kept[1]).all()


@pytest.mark.parametrize("pages,moves", [(70000, 33000), (70000, 32768), (40000, 32769), (5000, 5000), (100, 1)])
def test_compactions_of_many_pages(pages, moves):
    """Long lists; only the upper pages are in use."""
    import torch
    width = pages // 8
    b = Books(4, width, pages, 2, seed=pages)
    at = pages - 4 * (width - 1)
    for row in range(4):
        ids = list(range(at + row, pages, 4))[:width - 1]
        b.r.shuffle(ids)
        b.table[row][:len(ids)] = ids
        b.lens[row] = 2 * len(ids) - row % 2
    b.refs[:] = cache.count(b.table, b.lens, 2, pages)
    b.d_table.copy_(dev(b.table)), b.d_lens.copy_(dev(b.lens)), b.d_refs.copy_(dev(b.refs))
    b.compact(moves)
    b.fork([3, 2, 1, 0])
    b.compact(pages)
    assert torch.equal(b.d_refs > 0, torch.arange(pages, device="cuda") < int((b.d_refs > 0).sum()))
