"""Plain 64-bit definitions of the rotary positions and of attention over a
paged cache.

TEST INFRASTRUCTURE ONLY (see the package docstring). Literal: one pair, one
query and one visible position at a time in the formulas, numpy float64
throughout, no running maximum and no tiles.
"""
import numpy as np


def pair_axes(sections) -> np.ndarray:
    """The axis of each pair: sections[0] pairs of axis 0, then those of axis 1, ..."""
    return np.repeat(np.arange(len(sections)), sections)


def rope_ref(x, positions, inv_freq, sections, interleaved=False, inverse=False) -> np.ndarray:
    """x [T, H, D], positions [axes, T] integers, inv_freq [R]: float64 [T, H, D]."""
    x = np.asarray(x, dtype=np.float64)
    r = len(inv_freq)
    turn = np.asarray(positions)[pair_axes(sections)].astype(np.float64).T * np.asarray(inv_freq, dtype=np.float64)
    cos, sin = np.cos(turn)[:, None, :], np.sin(turn)[:, None, :]
    if inverse:
        sin = -sin
    i = np.arange(r)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def visible(n, kv, causal=True, window=0, sinks=0) -> np.ndarray:
    """bool [n, kv]: which positions each of a sequence's n last tokens sees."""
    p = (kv - n + np.arange(n))[:, None]
    j = np.arange(kv)[None, :]
    seen = np.ones((n, kv), dtype=bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def paged_attention_ref(q, k_cache, v_cache, page_table, kv_lens, q_starts, scale, causal=True, window=0, sinks=0):
    """(out [T, H, D], lse [T, H], spread [T, H, D], size [T, H]) in float64.

    spread = sum_j p_j |v_j| and size = |scale| max_j sum_d |q_d k_jd| over the
    visible positions: what the bounds of a finite-precision result go by.
    """
    q = np.asarray(q, dtype=np.float64)
    t, heads, d = q.shape
    page, kv_heads = k_cache.shape[1], k_cache.shape[2]
    out, spread = np.zeros((t, heads, d)), np.zeros((t, heads, d))
    lse, size = np.full((t, heads), -np.inf), np.zeros((t, heads))
    for b, kv in enumerate(kv_lens):
        s0, s1 = q_starts[b], q_starts[b + 1]
        seen = visible(s1 - s0, kv, causal, window, sinks)
        at = np.flatnonzero(seen.any(0))           # only these are looked up at all
        if at.size == 0:
            continue
        pages = np.asarray(page_table[b])[at // page]
        keys = np.asarray(k_cache[pages, at % page], dtype=np.float64)      # [len, kv_heads, d]
        values = np.asarray(v_cache[pages, at % page], dtype=np.float64)
        for i in range(s1 - s0):
            m = seen[i, at]
            if not m.any():
                continue
            for h in range(heads):
                kh, vh = keys[m, h // (heads // kv_heads)], values[m, h // (heads // kv_heads)]
                s = scale * (kh @ q[s0 + i, h])
                z = np.log(np.sum(np.exp(s - s.max()))) + s.max()
                w = np.exp(s - z)
                lse[s0 + i, h] = z
                out[s0 + i, h] = w @ vh
                spread[s0 + i, h] = w @ np.abs(vh)
                size[s0 + i, h] = abs(scale) * np.max(np.abs(kh) @ np.abs(q[s0 + i, h]))
    return out, lse, spread, size
