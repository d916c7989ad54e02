"""Attention with quantised projections over a paged cache: prompts in chunks, then
token by token, each step one projection, one rotation with its cache write and one
attention.

    python examples/attention_steps.py

Runs a batch of prompts of unlike lengths through one layer's attention on the
current GPU (synthetic weights), in chunks of at most 256 tokens, then generates a
few tokens for every sequence, and prints the time of a step.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from qkv_projection_gb300 import kaio  # noqa: E402


class PagedLayer:
    """One layer's attention: W4A16 projections, rotary positions, a paged cache.

    The projections give as many K/V heads as query heads. Pages are handed out in
    the order in which sequences grow into them.
    """

    def __init__(self, columns, heads, head_dim, sequences, pages, page_size=16, theta=10000.0, window=0, sinks=0,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = dict(device="cuda")
        n = heads * head_dim
        self.heads, self.head_dim, self.page_size = heads, head_dim, page_size
        self.window, self.sinks = window, sinks
        self.weights = [torch.randint(-2**31, 2**31 - 1, (columns // 8, n), dtype=torch.int32, generator=g, **dev)
                        for _ in range(3)]
        self.scales = [torch.full((columns // 128, n), 0.2 / math.sqrt(columns), dtype=torch.float16, **dev)
                       for _ in range(3)]
        self.inv_freq = (theta ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).float().cuda()
        shape = (pages, page_size, heads, head_dim)
        self.k_cache, self.v_cache = (torch.empty(shape, dtype=torch.float16, **dev) for _ in range(2))
        self.page_table = torch.full((sequences, pages), -1, dtype=torch.int32, **dev)
        self.free = list(range(pages))[::-1]
        self.lengths = [0] * sequences
        self.workspace = kaio.paged_attention_workspace()

    def step(self, x, new):
        """x f16 [sum(new), columns]: the next new[b] tokens of each sequence b, in order.
        Returns their attention outputs f16 [sum(new), heads * head_dim]."""
        positions, slots, starts = [], [], [0]
        for b, n in enumerate(new):
            for p in range(self.lengths[b], self.lengths[b] + n):
                if p % self.page_size == 0:
                    self.page_table[b, p // self.page_size] = self.free.pop()
            positions += range(self.lengths[b], self.lengths[b] + n)
            self.lengths[b] += n
            starts.append(starts[-1] + n)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        positions, starts, lengths = ints(positions), ints(starts), ints(self.lengths)
        owner = torch.repeat_interleave(torch.arange(len(new), device="cuda"), (starts[1:] - starts[:-1]).long())
        slots = self.page_table[owner, positions // self.page_size] * self.page_size + positions % self.page_size

        rows = (x.shape[0], self.heads, self.head_dim)
        q, k, v = (t.view(rows) for t in kaio.qkv_project_int4(x, *self.weights, *self.scales))
        kaio.rope_append(q, k, v, positions, self.inv_freq, self.k_cache, self.v_cache, slots, q_out=q)
        out = kaio.paged_attention(q, self.k_cache, self.v_cache, self.page_table, lengths, starts, max_new=max(new),
                                   window=self.window, sinks=self.sinks, workspace=self.workspace)
        return out.view(x.shape[0], -1)


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
          f"{begin.elapsed_time(end) / 20 * 1e3:.0f} us a step (with the bookkeeping on the host)")


if __name__ == "__main__":
    main()
