"""Arguments of the rotary and attention calls that are no integers, or none that the
library's fields hold, are refused by name; the library refuses the rest (no GPU)."""
import pytest
import torch

from qkv_projection_gb300 import kaio

F16, I32 = torch.float16, torch.int32


@pytest.fixture(autouse=True)
def by_python(monkeypatch):
    monkeypatch.setattr(kaio, "_host", lambda: False)
    monkeypatch.setattr(kaio, "_host_module", False)
    monkeypatch.setattr(kaio, "_strides", lambda t, *a: t.stride())       # CPU tensors stand in
    monkeypatch.setattr(kaio, "_current_raw_stream", lambda device: 0)


class Workspace:
    is_cuda, dtype = True, torch.uint8
    is_contiguous, data_ptr, numel = (lambda self: True), (lambda self: 1 << 40), (lambda self: 64)


def attend(d=64, **kw):
    q, cache = torch.zeros(2, 4, d, dtype=F16), torch.zeros(3, 16, 2, d, dtype=F16)
    kw.setdefault("workspace", Workspace())
    return kaio.paged_attention(q, cache, cache, torch.zeros(2, 1, dtype=I32), torch.zeros(2, dtype=I32), **kw)


@pytest.mark.parametrize("name", ["window", "sinks", "max_new"])
def test_integers_of_attention(name):
    for v in (2 ** 31, -2 ** 31 - 1, 1 << 80):
        with pytest.raises(ValueError, match=name):
            attend(**{name: v})
    for v in (1.5, "3", object()):
        with pytest.raises(TypeError, match=name):
            attend(**{name: v})


def test_scale_and_dim():
    for scale in (1e39, float("inf"), float("nan")):
        with pytest.raises(kaio.KaioError, match="scale"):
            attend(scale=scale)
    with pytest.raises(TypeError):
        attend(scale="x")
    with pytest.raises(kaio.KaioError, match="dim"):
        attend(d=0)


def test_workspace_that_is_no_tensor():
    for other in (3, b"12", object()):
        with pytest.raises(ValueError, match="workspace"):
            attend(workspace=other)


def test_sections_and_sizes():
    x, pos, freq = torch.zeros(2, 4, 64, dtype=F16), torch.zeros(1, 2, dtype=I32), torch.zeros(32)
    for v, error in ((1 << 40, ValueError), (1.5, TypeError), (None, TypeError)):
        with pytest.raises(error, match="sections"):
            kaio.rope(x, pos, freq, sections=(v,))
        with pytest.raises(error, match="sections"):
            kaio.rope_append(x, x, x, pos, freq, x[None], x[None], pos[0], sections=(v,))
    many = x[:1].expand(1 << 31, 4, 64)
    with pytest.raises(ValueError, match="size"):
        kaio.rope(many, pos[:, :1].expand(1, 1 << 31), freq, out=many)
