"""The books' oracle against what has to hold of any books: references that agree with the
table, contents that follow their pages (no GPU)."""
import random

import pytest

from oracle import cache


class Books:
    """Sequences that write a number of their own into every position."""

    def __init__(self, batch, width, pages, page):
        self.page, self.pages = page, pages
        self.refs, self.table, self.lens = [0] * pages, [[-5] * width for _ in range(batch)], [0] * batch
        self.data = [[None] * page for _ in range(pages)]
        self.want = [[] for _ in range(batch)]
        self.next = 0

    def check(self):
        assert self.refs == cache.count(self.table, self.lens, self.page, self.pages)
        for row, n, want in zip(self.table, self.lens, self.want):
            assert [self.data[row[i // self.page]][i % self.page] for i in range(n)] == want

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            if s >= 0:
                self.data[d] = list(self.data[s])

    def append(self, new):
        starts = [sum(new[:i]) for i in range(len(new) + 1)]
        slots, src, dst = cache.append(self.refs, self.table, self.lens, starts, starts[-1], self.page)
        self.copy(src, dst)
        for b, n in enumerate(new):
            mine = slots[starts[b]:starts[b + 1]]
            assert all(s >= 0 for s in mine) or all(s < 0 for s in mine)
            for s in mine:
                if s >= 0:
                    self.data[s // self.page][s % self.page] = self.next
                    self.want[b].append(self.next)
                    self.next += 1


@pytest.mark.parametrize("seed", range(6))
def test_books_stay_consistent(seed):
    r = random.Random(seed)
    batch, page = r.randint(1, 6), r.choice([1, 3, 4])
    b = Books(batch, 12, r.randint(10, 40), page)
    for _ in range(60):
        what = r.choice(["append", "append", "fork", "truncate", "compact"])
        if what == "append":
            b.append([r.randint(0, 7) for _ in range(batch)])
        elif what == "fork":
            parents = [r.randint(-1, batch) for _ in range(batch)]
            cache.fork(b.refs, b.table, b.lens, parents, page)
            b.want = [list(b.want[a if 0 <= a < batch else i]) for i, a in enumerate(parents)]
        elif what == "truncate":
            new = [r.randint(-2, 20) for _ in range(batch)]
            cache.truncate(b.refs, b.table, b.lens, new, page)
            b.want = [w[:max(n, 0)] for w, n in zip(b.want, new)]
        else:
            moves = r.choice([0, 1, 3, 50])
            src, dst = cache.compact(b.refs, b.table, b.lens, page, moves)
            b.copy(src, dst)
            if moves == 50:
                used = sum(x > 0 for x in b.refs)
                assert all(x > 0 for x in b.refs[:used])
        b.check()


def test_copy_pages_leaves_out_pages_outside():
    c = [[1, 2, 3], [4, 5, 6]]
    cache.copy_pages(c, [0, -1, 3, 1], [2, 1, 0, 9])
    assert c == [[1, 2, 1], [4, 5, 4]]
