"""Attention with quantised projections over a paged cache: prompts in chunks, then
token by token, each step pages for the new tokens, one projection, one rotation with its
cache write and one attention.

    python examples/attention_steps.py

Runs a batch of prompts of unlike lengths through one layer's attention on the
current GPU (synthetic weights), in chunks of at most 256 tokens, then generates a
few tokens for every sequence, forks one into all rows, cuts what was drafted, compacts
the cache, and prints the time of a step.
"""
import math
import os
import sys
from collections import Counter

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from qkv_projection_gb300 import kaio  # noqa: E402


class PagedLayer:
    """One layer's attention: W4A16 projections, rotary positions, a paged cache.

    The projections give as many K/V heads as query heads. Which sequence holds which
    pages is kept on the GPU (page_refs, page_table, kv_lens). `lengths` follows on the host, and so does
    how many pages are left, under numbers of the host's own (`held`: the pages of each row, `holders`: how
    many hold each): a step for which there is no room is refused before anything is sent, since on
    the GPU a row that does not fit takes nothing, silently.
    softcap and slopes (f32 [heads]) are those of ``kaio.paged_attention``.
    """

    def __init__(self, columns, heads, head_dim, sequences, pages, page_size=16, theta=10000.0, window=0, sinks=0,
                 seed=0, softcap=0.0, slopes=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = dict(device="cuda")
        n = heads * head_dim
        self.heads, self.head_dim, self.page_size = heads, head_dim, page_size
        self.window, self.sinks, self.softcap, self.slopes = window, sinks, softcap, slopes
        self.weights = [torch.randint(-2**31, 2**31 - 1, (columns // 8, n), dtype=torch.int32, generator=g, **dev)
                        for _ in range(3)]
        self.scales = [torch.full((columns // 128, n), 0.2 / math.sqrt(columns), dtype=torch.float16, **dev)
                       for _ in range(3)]
        self.inv_freq = (theta ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).float().cuda()
        shape = (pages, page_size, heads, head_dim)
        self.k_cache, self.v_cache = (torch.empty(shape, dtype=torch.float16, **dev) for _ in range(2))
        self.page_refs = torch.zeros(pages, dtype=torch.int32, **dev)
        self.page_table = torch.full((sequences, pages), -1, dtype=torch.int32, **dev)
        self.kv_lens = torch.zeros(sequences, dtype=torch.int32, **dev)
        self.lengths = [0] * sequences
        self.held, self.holders, self.named = [[] for _ in range(sequences)], Counter(), 0
        self.workspace = kaio.paged_attention_workspace()

    def step(self, x, new):
        """x f16 [sum(new), columns]: the next new[b] tokens of each sequence b, in order.
        Returns their attention outputs f16 [sum(new), heads * head_dim]."""
        self.take(new)
        positions, starts = [], [0]
        for b, n in enumerate(new):
            positions += range(self.lengths[b], self.lengths[b] + n)
            self.lengths[b] += n
            starts.append(starts[-1] + n)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        positions, starts = ints(positions), ints(starts)
        # pages for the new tokens; where a last page is shared, its row gets a copy of its own
        slots, src, dst = kaio.cache_append(*self.books(), starts, x.shape[0], self.page_size)
        kaio.cache_copy_pages((self.k_cache, self.v_cache), src, dst)

        rows = (x.shape[0], self.heads, self.head_dim)
        q, k, v = (t.view(rows) for t in kaio.qkv_project_int4(x, *self.weights, *self.scales))
        kaio.rope_append(q, k, v, positions, self.inv_freq, self.k_cache, self.v_cache, slots, q_out=q)
        out = kaio.paged_attention(q, self.k_cache, self.v_cache, self.page_table, self.kv_lens, starts, max_new=max(new),
                                   window=self.window, sinks=self.sinks, workspace=self.workspace, softcap=self.softcap,
                                   slopes=self.slopes)
        return out.view(x.shape[0], -1)

    def take(self, new):
        """Pages for new[b] more tokens of each row, as cache_append gives them out."""
        places = lambda n: -(-n // self.page_size)  # noqa: E731
        own = [int(n > 0 and self.lengths[b] % self.page_size > 0 and self.holders[self.held[b][-1]] > 1)
               for b, n in enumerate(new)]                 # a shared last page is replaced
        more = [places(self.lengths[b] + n) - len(self.held[b]) for b, n in enumerate(new)]
        pages, rows = self.page_refs.numel(), self.page_table.shape[1]
        if sum(own) + sum(more) > pages - len(self.holders) or any(m + len(h) > rows for m, h in zip(more, self.held)):
            raise RuntimeError(f"the cache is full: {sum(own) + sum(more)} pages more, {pages - len(self.holders)} of {pages} left")
        for row, o, m in zip(self.held, own, more):
            if o:
                self.holders[row.pop()] -= 1
            made = range(self.named, self.named + o + m)
            row += made
            self.holders.update(made)
            self.named = made.stop
        if any(own):
            self.holders = +self.holders                   # (without those that nobody holds any more)

    def count(self):
        self.holders = Counter(p for row in self.held for p in row)

    def books(self):
        return self.page_refs, self.page_table, self.kv_lens

    def fork(self, parents):
        """Row b goes on from where row parents[b] stands; they share their pages. A parent that is no row leaves its row."""
        kaio.cache_fork(*self.books(), torch.tensor(parents, dtype=torch.int32, device="cuda"), self.page_size)
        parents = [p if 0 <= p < len(self.lengths) else b for b, p in enumerate(parents)]
        self.lengths = [self.lengths[p] for p in parents]
        self.held = [list(self.held[p]) for p in parents]
        self.count()

    def truncate(self, lengths):
        """Drops what each row has past these lengths (drafts that were refused; 0: the sequence is done)."""
        kaio.cache_truncate(*self.books(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), self.page_size)
        self.lengths = [min(a, max(b, 0)) for a, b in zip(self.lengths, lengths)]
        self.held = [row[:-(-n // self.page_size)] for row, n in zip(self.held, self.lengths)]
        self.count()

    def compact(self):
        """Moves all pages in use to the beginning of the cache."""
        pages = self.page_refs.numel()
        src, dst = kaio.cache_compact(*self.books(), self.page_size, (pages + 1) // 2)
        kaio.cache_copy_pages((self.k_cache, self.v_cache), src, dst)


def main():
    columns, heads, head_dim, chunk = 4096, 32, 128, 256
    prompts = [700, 45, 1300, 256]
    layer = PagedLayer(columns, heads, head_dim, len(prompts), pages=1024)
    left = list(prompts)
    while any(left):
        new = [min(n, chunk) for n in left]
        out = layer.step(torch.randn(sum(new), columns, dtype=torch.float16, device="cuda"), new)
        left = [a - b for a, b in zip(left, new)]
        print(f"prompt step of {new} tokens: output {tuple(out.shape)}")
    ones = [1] * len(prompts)
    x = torch.randn(len(prompts), columns, dtype=torch.float16, device="cuda")
    for _ in range(3):
        layer.step(x, ones)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        layer.step(x, ones)
    end.record()
    kaio.device_status()
    print(f"one token for each of {len(prompts)} sequences of {layer.lengths} positions: "
          f"{begin.elapsed_time(end) / 20 * 1e3:.0f} us a step (positions counted on the host)")

    layer.fork([0] * len(prompts))                         # four samples of the longest prompt
    layer.step(x, ones)
    layer.step(torch.cat([x] * 4), [4] * len(prompts))     # four drafted tokens each, of which one to four stay
    layer.truncate([n - b for b, n in enumerate(layer.lengths)])
    layer.compact()
    out = layer.step(x, ones)
    kaio.device_status()
    print(f"forked, drafted, cut and compacted: {layer.lengths} positions in {int((layer.page_refs > 0).sum())} pages, "
          f"output {tuple(out.shape)}")


if __name__ == "__main__":
    main()
