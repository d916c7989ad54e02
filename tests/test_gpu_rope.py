"""Rotary positions and the fused cache write against the 64-bit definition.

Tolerance: the result is an f32 value rounded once to p significant bits, so it
is within 2^-p of its size (and half the smallest subnormal, 2^-25, in f16) of
that f32 value. The f32 value is off by two products and a sum (3 * 2^-24 of
|x0| + |x1|) and by the sine and cosine: the angle is held to 2^-25 turns and
rounded from there to f32, at most 2^-24 turns = 3.8e-7 radians, and the sine's
own error is a few 2^-24. Together below 1e-6 * (|x0| + |x1|).
"""
import numpy as np
import pytest

from oracle.attention import rope_ref
from qkv_projection_gb300 import kaio

pytestmark = pytest.mark.gpu

BITS = {"float16": 11, "bfloat16": 8}


def _inputs(t, h, d, pairs, axes, dtype, seed=0, top=5000):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(t, h, d, device="cuda", generator=g).to(getattr(torch, dtype))
    pos = torch.randint(0, top, (axes, t), device="cuda", generator=g, dtype=torch.int32)
    inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
    sections = [pairs // axes] * axes
    sections[-1] += pairs - sum(sections)
    return x, pos, inv, tuple(sections)


def _host(t):
    return t.double().cpu().numpy()


def _check(got, x, pos, inv, sections, interleaved, inverse, dtype, angle=1.01e-6):
    x64 = _host(x)
    ref = rope_ref(x64, pos.cpu().numpy(), inv.double().cpu().numpy(), sections, interleaved, inverse)
    r = inv.shape[0]
    size = np.abs(x64).copy()
    i = np.arange(r)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    size[..., a] = size[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    bound = 2.0 ** -BITS[dtype] * np.abs(ref) + angle * size + 2.0 ** -25
    err = np.abs(_host(got) - ref)
    assert np.all(err <= bound), (err - bound).max()
    np.testing.assert_array_equal(_host(got)[..., 2 * r:], x64[..., 2 * r:])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,h,d,pairs,axes", [
    (1, 1, 8, 1, 1), (1, 32, 128, 64, 1), (3, 5, 64, 32, 3), (7, 3, 80, 40, 2), (5, 2, 96, 33, 3),
    (2, 4, 128, 52, 4), (130, 2, 256, 128, 2), (4900, 2, 72, 20, 1), (4901, 1, 40, 7, 2),
])
def test_rope_and_its_gradient(t, h, d, pairs, axes, interleaved, dtype):
    x, pos, inv, sections = _inputs(t, h, d, pairs, axes, dtype, seed=t + d)
    for inverse in (False, True):
        got = kaio.rope(x, pos, inv, sections=sections, interleaved=interleaved, inverse=inverse)
        _check(got, x, pos, inv, sections, interleaved, inverse, dtype)


def test_gradient_against_differences():
    """dx = inverse(dy): along random directions u, the difference quotient of
    sum(dy * rope(x)) is sum(dx * u). The rotation is linear, so the quotient is
    exact up to rounding: three results rounded to 2^-11 of values whose products
    add up like a random walk, over a step of 1; 64 * 5 standard deviations."""
    import torch
    x, pos, inv, sections = _inputs(64, 4, 128, 64, 3, "float16", seed=5)
    dy = torch.randn_like(x)
    dx = kaio.rope(dy, pos, inv, sections=sections, inverse=True).double()
    for seed in range(3):
        u = torch.randn(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).half()
        up = kaio.rope((x + u), pos, inv, sections=sections).double()
        base = kaio.rope(x, pos, inv, sections=sections).double()
        step = (x + u).double() - x.double()
        quotient = ((up - base) * dy.double()).sum()
        direct = (dx * step).sum()
        sigma = 3 * 2.0 ** -11 * x.numel() ** 0.5 * 2
        assert abs(quotient - direct) < 5 * sigma


def test_large_positions_are_exact():
    """Positions up to 2^31 - 1 and negative ones: the bound does not grow with them."""
    import torch
    x, _, inv, _ = _inputs(6, 2, 128, 64, 1, "float16", seed=9)
    pos = torch.tensor([[0, -1, 100003, 16777217, 2**31 - 1, -2**31]], dtype=torch.int32, device="cuda")
    # besides: the definition's own angle is good to 2^-53 * 2^31 = 2.4e-7 radians, and the frequency
    # in turns, held to 2 * 2^-53 of its size, to 4.2e-7 radians at 2^31 / 2 pi turns
    _check(kaio.rope(x, pos, inv), x, pos, inv, (64,), False, False, "float16", angle=2e-6)


def test_strided_views_in_place_and_other_stream():
    import torch
    x, pos, inv, _ = _inputs(33, 12, 64, 32, 1, "float16", seed=3)
    packed = x.view(33, 3, 4, 64).transpose(1, 2)                       # [T, 4, 3, D], strided
    view = packed[:, :, 1]
    got = kaio.rope(view, pos[0], inv)
    _check(got, view, pos, inv, (32,), False, False, "float16")
    out = torch.zeros(33, 4, 2, 64, dtype=torch.float16, device="cuda")
    kaio.rope(view, pos, inv, out=out[:, :, 1])
    assert torch.equal(out[:, :, 1], got) and not out[:, :, 0].any()
    broadcast = x[:, :1].expand(33, 5, 64)
    _check(kaio.rope(broadcast, pos, inv), broadcast, pos, inv, (32,), False, False, "float16")
    for pairs in (32, 27):                                              # vector and scalar forms
        y = x.clone()
        want = kaio.rope(x, pos, inv[:pairs])
        assert kaio.rope(y, pos, inv[:pairs], out=y) is y and torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kaio.rope(view, pos[0], inv, stream=side)
    side.synchronize()
    assert torch.equal(other, got)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t,h,kh,d,pairs,page,layout", [
    (1, 32, 32, 128, 64, 16, "slots_first"), (45, 6, 2, 64, 32, 16, "heads_first"),
    (45, 6, 3, 80, 21, 7, "slots_first"), (4870, 3, 1, 128, 64, 64, "one_buffer"),
])
def test_append(t, h, kh, d, pairs, page, layout, dtype):
    import torch
    q, pos, inv, sections = _inputs(t, h, d, pairs, 3, dtype, seed=t + h)
    k, v = _inputs(t, kh, d, pairs, 1, dtype, seed=1)[0], _inputs(t, kh, d, pairs, 1, dtype, seed=2)[0]
    pages = -(-t // page) + 2
    td = getattr(torch, dtype)
    if layout == "heads_first":
        kc, vc = (torch.full((pages, kh, page, d), 7.0, dtype=td, device="cuda").transpose(1, 2) for _ in range(2))
    elif layout == "one_buffer":
        both = torch.full((pages, 2, page, kh, d), 7.0, dtype=td, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = (torch.full((pages, page, kh, d), 7.0, dtype=td, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:t].to(torch.int32)
    if t > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, 2**31 - 1      # not stored
    got = kaio.rope_append(q, k, v, pos, inv, kc, vc, slots, sections=sections)
    _check(got, q, pos, inv, sections, False, False, dtype)
    real = (slots >= 0) & (slots < pages * page)
    at = slots[real].long()
    at = (at // page, at % page)
    _check(kc[at], k[real], pos[:, real], inv, sections, False, False, dtype)
    assert torch.equal(vc[at], v[real])
    untouched = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    untouched[at] = False
    assert (kc[untouched] == 7).all() and (vc[untouched] == 7).all()
    kc2, vc2 = kc.clone(), vc.clone()
    same = kaio.rope_append(q, k, v, pos, inv, kc2, vc2, slots, sections=sections, q_out=q)
    assert same is q and torch.equal(q, got) and torch.equal(kc2, kc)


def test_no_tokens_and_an_empty_cache():
    import torch
    x, pos, inv, _ = _inputs(2, 2, 64, 32, 1, "float16")
    assert kaio.rope(x[:0], pos[:, :0], inv).shape == (0, 2, 64)
    cache = torch.empty(0, 16, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert torch.equal(kaio.rope_append(x, x, x, pos, inv, cache, cache.clone(), slots), kaio.rope(x, pos, inv))


def test_refusals():
    import torch
    x, pos, inv, _ = _inputs(4, 2, 64, 32, 2, "float16")
    with pytest.raises(ValueError, match="sections"):
        kaio.rope(x, pos, inv)
    with pytest.raises(kaio.KaioError, match="sections sum"):
        kaio.rope(x, pos, inv, sections=(16, 15))
    with pytest.raises(kaio.KaioError, match="pairs"):
        kaio.rope(x, pos[0], torch.ones(33, device="cuda"))
    both = x.repeat(2, 1, 1)
    with pytest.raises(kaio.KaioError, match="overlap"):
        kaio.rope(both[:4], pos[0], inv, out=both[2:6])
    with pytest.raises(TypeError, match="float16 or"):
        kaio.rope(x.float(), pos[0], inv)
    with pytest.raises(TypeError, match="positions"):
        kaio.rope(x, pos[0].long(), inv)
    with pytest.raises(ValueError, match="dense last"):
        kaio.rope(x.transpose(1, 2), pos[0], inv)
    with pytest.raises(ValueError, match="gradient"):
        kaio.rope(x.clone().requires_grad_(), pos[0], inv)
    with pytest.raises(kaio.KaioError, match="MISALIGNED"):
        kaio.rope(x.view(-1)[4:4 + 256].view(2, 2, 64), pos[0, :2].contiguous(), inv)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(kaio.KaioError, match="k_cache and v_cache"):
        kaio.rope_append(x, x, x, pos[0], inv, cache, cache, slots)
    with pytest.raises(ValueError, match="v_cache"):
        kaio.rope_append(x, x, x, pos[0], inv, cache, cache[:1], slots)
