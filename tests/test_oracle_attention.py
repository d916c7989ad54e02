"""The 64-bit definitions of rotary positions and paged attention, pinned to
facts that do not come from them: complex multiplication, orthogonality,
differences, hand-written masks and closed forms. No GPU."""
import numpy as np
import pytest

from oracle.attention import paged_attention_ref, pair_axes, rope_ref, visible


def _rng(seed=0):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_multiplication_by_a_unit_complex_number(interleaved):
    rng = _rng()
    x = rng.standard_normal((5, 2, 10))
    pos = rng.integers(0, 1000, (2, 5))
    inv = np.array([1.0, 0.3, 0.01, 0.002], dtype=np.float32)
    y = rope_ref(x, pos, inv, (1, 3), interleaved)
    for i, axis in enumerate((0, 1, 1, 1)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axis] * np.float64(inv[i]))[:, None]
        np.testing.assert_allclose(y[..., a], z.real, rtol=0, atol=1e-13)
        np.testing.assert_allclose(y[..., b], z.imag, rtol=0, atol=1e-13)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])


def test_rope_scores_depend_on_the_distance_alone():
    q, k = _rng(1).standard_normal((2, 1, 1, 8))
    inv = 100.0 ** (-np.arange(4) / 4)
    dots = [np.sum(rope_ref(q, [[p]], inv, (4,)) * rope_ref(k, [[p - 7]], inv, (4,))) for p in (7, 50, 12345)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_rope_gradient_is_the_inverse_rotation_by_differences():
    rng = _rng(2)
    x, g = rng.standard_normal((2, 3, 2, 6))
    pos, inv = rng.integers(0, 99, (1, 3)), np.array([0.7, 0.05])
    dx = rope_ref(g, pos, inv, (2,), inverse=True)
    for at in np.ndindex(x.shape):
        h = np.zeros_like(x)
        h[at] = 1e-4
        diff = np.sum(g * (rope_ref(x + h, pos, inv, (2,)) - rope_ref(x - h, pos, inv, (2,)))) / 2e-4
        assert abs(diff - dx[at]) < 1e-9
    np.testing.assert_allclose(rope_ref(rope_ref(x, pos, inv, (2,)), pos, inv, (2,), inverse=True), x, atol=1e-14)


def test_pair_axes():
    assert pair_axes((2, 0, 3)).tolist() == [0, 0, 2, 2, 2]


def test_visible_by_hand():
    assert visible(2, 4).astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert visible(2, 4, causal=False).all()
    assert visible(1, 6, window=2).astype(int).tolist() == [[0, 0, 0, 0, 1, 1]]
    assert visible(2, 6, window=2, sinks=1).astype(int).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert visible(3, 2).astype(int).tolist() == [[0, 0], [1, 0], [1, 1]]       # the first token stands before all


def _cache(rng, lens, page, kv_heads, d):
    per = [-(-n // page) for n in lens]
    pages = rng.permutation(sum(per) + 1)
    table = np.full((len(lens), max(max(per), 1)), -1)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = pages[at:at + n]
        at += n
    return rng.standard_normal((2, sum(per) + 1, page, kv_heads, d)), table


def test_attention_closed_forms():
    rng = _rng(3)
    lens = [5, 1]
    (kc, vc), table = _cache(rng, lens, 4, 2, 3)
    # scale 0: plain means of the visible values, lse = ln of their number
    out, lse, _, _ = paged_attention_ref(np.ones((3, 4, 3)), kc, vc, table, lens, [0, 2, 3], 0.0)
    flat = lambda b, n: np.stack([vc[table[b, j // 4], j % 4] for j in range(n)])  # noqa: E731
    for row, (b, n) in enumerate(((0, 4), (0, 5), (1, 1))):
        np.testing.assert_allclose(out[row], np.repeat(flat(b, n).mean(0), 2, axis=0), atol=1e-15)
        np.testing.assert_allclose(lse[row], np.log(n), atol=1e-15)
    # one key with all the weight
    kc[:] = 0
    kc[table[0, 0], 2] = 100.0
    out, lse, _, _ = paged_attention_ref(np.ones((1, 4, 3)), kc, vc, table[:1], [5], [0, 1], 1.0)
    np.testing.assert_allclose(out[0], np.repeat(vc[table[0, 0], 2], 2, axis=0), atol=1e-100)
    np.testing.assert_allclose(lse[0], 300.0)


def test_attention_of_nothing():
    out, lse, _, _ = paged_attention_ref(np.ones((3, 2, 8)), np.ones((1, 16, 1, 8)), np.ones((1, 16, 1, 8)),
                                         [[0], [0]], [0, 1], [0, 1, 3], 1.0)
    assert not out[:2].any() and np.isneginf(lse[:2]).all()
    np.testing.assert_allclose(out[2], 1.0)
