"""Attention over a paged cache where the division of its work decides what runs: whole
items of two halves in numbers, tiles of half the rows, items of few and of many rows in
one line, and shares whose boundaries fall on, near and between the ends of items. The
tolerance is that of test_gpu_paged_attention.py."""
import pytest

from test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu


def twice(p, **mask):
    first = p.verify(**mask)
    again = p.run(**mask)
    assert all((a == b).all() for a, b in zip(first, again))


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("float16", 64), ("float16", 72)])
@pytest.mark.parametrize("mask", [dict(), dict(window=100, sinks=5), dict(window=130), dict(causal=False)])
def test_many_whole_items_of_two_halves(mask, d, dtype):
    # 8 K/V heads x 2 tiles x 12 sequences: more than half as many items as CTAs
    lens = [(40, 40 + 29 * i) for i in range(12)]
    twice(Problem(lens, 64, 8, d, 32, dtype, seed=3), **mask)


@pytest.mark.parametrize("mask", [dict(), dict(window=300, sinks=130), dict(causal=False)])
@pytest.mark.parametrize("n,kv", [(129, 129), (100, 1000), (257, 2040), (33, 500)])
def test_few_items_in_tiles_of_half_the_rows(n, kv, mask):
    twice(Problem([(n, kv), (3, 5), (0, 9)], 5, 1, 64, 16, "bfloat16", seed=n), **mask)


@pytest.mark.parametrize("mask", [dict(), dict(window=2500, sinks=3)])
def test_few_and_many_rows_in_one_line(mask):
    lens = [(1, 2200), (90, 3100), (1, 1), (1, 5000), (4, 2177), (60, 60), (1, 2047), (33, 2600), (1, 4097)]
    twice(Problem(lens, 8, 2, 128, 64, "float16", seed=5), **mask)


@pytest.mark.parametrize("kv", [2049, 2176, 2300, 3500, 6000])
@pytest.mark.parametrize("n,sequences,heads", [(9, 3, 8), (65, 2, 8), (40, 7, 16)])
def test_boundaries_near_the_ends_of_items(n, sequences, heads, kv):
    twice(Problem([(n, kv + i) for i in range(sequences)], heads, heads // 4, 64, 32, "float16", seed=kv))


@pytest.mark.parametrize("kv", [512, 513, 577, 1037, 1300])
@pytest.mark.parametrize("sequences,heads", [(1, 32), (5, 12), (30, 16), (64, 8)])
def test_boundaries_near_the_ends_of_items_of_single_tokens(sequences, heads, kv):
    twice(Problem([(1, kv + 3 * i) for i in range(sequences)], heads, heads // 2, 64, 16, "bfloat16", seed=kv))
