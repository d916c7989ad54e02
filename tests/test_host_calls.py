"""The one-step host path of the rotary and attention calls against the code in Python:
it leaves to Python whatever it does not take (no GPU), and gives the same results."""
import math

import pytest
import torch

from qkv_projection_gb300 import kaio


@pytest.fixture(scope="module")
def host():
    module = kaio._host()
    if not module:
        pytest.skip("built without Python's or torch's headers")
    return module


def tensors(device, dtype=torch.float16, t=6, h=4, kh=2, d=64, pages=5, page=16):
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(device)   # noqa: E731
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=device)   # noqa: E731
    return dict(q=r(t, h, d), k=r(t, kh, d), v=r(t, kh, d), kc=r(pages, page, kh, d), vc=r(pages, page, kh, d),
                pos=i(list(range(20, 20 + t))), pos2=i([list(range(t)), list(range(5, 5 + t))]),
                freq=torch.logspace(0, -3, d // 2).to(device), slots=i([3, -1, 17, 40, 5, 70][:t]),
                table=i([[4, 0, 2], [1, 3, 0]]), lens=i([37, 20]), starts=i([0, 2, t]))


def test_leaves_what_it_does_not_take(host):
    a = tensors("cpu")
    rope = (a["q"], a["pos"], a["freq"], None, False, False, None, None)
    append = (a["q"], a["k"], a["v"], a["pos"], a["freq"], a["kc"], a["vc"], a["slots"], None, False, None, None)
    attend = (a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"], None, None, True, 0, 0,
              torch.zeros(64, dtype=torch.uint8), None, False, None, None)
    for call, args in ((host.rope, rope), (host.rope_append, append), (host.paged_attention, attend)):
        assert call(*args) is None                    # on the CPU
        assert call(*args[:-1]) is None               # too few
        assert call() is None
        for i in range(len(args)):
            for other in (None, 3, "x", object(), torch.zeros(2), float("nan"), 1 << 80):
                assert call(*args[:i], other, *args[i + 1:]) is None


def test_bind_takes_three_addresses(host):
    with pytest.raises(TypeError):
        host.bind(1)
    with pytest.raises(TypeError):
        host.bind("a", 2, 3)


def both(monkeypatch, run):
    """The results of run() by the host module and by Python."""
    assert kaio._host()
    a = run()
    with monkeypatch.context() as m:
        m.setattr(kaio, "_host", lambda: False)
        m.setattr(kaio, "_host_module", False)
        b = run()
    return a, b


def same(a, b):
    for x, y in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride()
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t", [0, 1, 6])
def test_rope_the_same_either_way(host, monkeypatch, dtype, t):
    a = tensors("cuda", dtype)
    cut = lambda n: a[n][:t]   # noqa: E731
    q, k, v, slots, pos = cut("q"), cut("k"), cut("v"), cut("slots"), cut("pos")
    for kw in (dict(), dict(interleaved=True), dict(inverse=True), dict(sections=[32])):
        same(*both(monkeypatch, lambda: kaio.rope(q, pos, a["freq"], **kw)))
    same(*both(monkeypatch, lambda: kaio.rope(q, a["pos2"][:, :t], a["freq"], sections=(20, 12))))
    wide = torch.zeros(t, 4, 96, dtype=dtype, device="cuda")[..., :64]
    same(*both(monkeypatch, lambda: kaio.rope(q, pos, a["freq"], out=wide).clone()))
    assert kaio.rope(q, pos, a["freq"], out=wide) is wide

    def append():
        kc, vc = a["kc"].clone(), a["vc"].clone()
        out = kaio.rope_append(q, k, v, pos, a["freq"], kc, vc, slots)
        return out, kc, vc
    same(*both(monkeypatch, append))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attention_the_same_either_way(host, monkeypatch, dtype):
    a = tensors("cuda", dtype)
    ws = kaio.paged_attention_workspace()
    args = (a["q"], a["kc"], a["vc"], a["table"], a["lens"])
    for kw in (dict(), dict(max_new=4), dict(scale=0.3), dict(causal=False), dict(window=7, sinks=3),
               dict(return_lse=True), dict(out=torch.empty_like(a["q"])),
               dict(lse=torch.empty(6, 4, device="cuda"), return_lse=True)):
        same(*both(monkeypatch, lambda: kaio.paged_attention(*args, a["starts"], workspace=ws, **kw)))
    one = (a["q"][:2],) + args[1:]
    same(*both(monkeypatch, lambda: kaio.paged_attention(*one, workspace=ws)))
    heads_first = a["kc"].transpose(1, 2).contiguous().transpose(1, 2)
    same(*both(monkeypatch, lambda: kaio.paged_attention(one[0], heads_first, *args[2:], workspace=ws)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kaio.paged_attention(*args, a["starts"], workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, kaio.paged_attention(*args, a["starts"], workspace=ws))


@pytest.mark.gpu
def test_refusals_say_the_same(host, monkeypatch):
    a = tensors("cuda")
    ws = kaio.paged_attention_workspace()
    grad = a["q"].clone().requires_grad_()
    calls = [lambda: kaio.rope(grad, a["pos"], a["freq"]), lambda: kaio.rope(a["q"], a["pos2"], a["freq"]),
             lambda: kaio.rope(a["q"], a["pos"], a["freq"][:0]), lambda: kaio.rope(a["q"].float(), a["pos"], a["freq"]),
             lambda: kaio.rope_append(a["q"], a["k"], a["v"][1:], a["pos"], a["freq"], a["kc"], a["vc"], a["slots"]),
             lambda: kaio.rope_append(a["q"], a["k"], a["v"], a["pos"], a["freq"], a["kc"], a["kc"], a["slots"]),
             lambda: kaio.paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"].long(),
                                          workspace=ws),
             lambda: kaio.paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"], window=-1,
                                          workspace=ws),
             lambda: kaio.paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"],
                                          workspace=ws[:64])]
    for call in calls:
        with pytest.raises((TypeError, ValueError, kaio.KaioError)) as one:
            call()
        with monkeypatch.context() as m:
            m.setattr(kaio, "_host", lambda: False)
            m.setattr(kaio, "_host_module", False)
            with pytest.raises((TypeError, ValueError, kaio.KaioError)) as other:
                call()
        assert type(one.value) is type(other.value) and str(one.value) == str(other.value)
    assert math.isfinite(float(kaio.rope(a["q"], a["pos"], a["freq"]).float().sum()))
