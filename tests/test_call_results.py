"""Results that the rotary and attention calls make for themselves belong to the call's
stream: on the current stream's memory that stream's earlier work might not be done, and
its later work would get the memory while the kernel still writes."""
import contextlib

import pytest
import torch

from qkv_projection_gb300 import kaio


class Library:
    """Launches nothing."""

    def __getattr__(self, name):
        return lambda *args: kaio.KAIO_OK


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


def test_are_made_on_the_stream_that_the_kernel_runs_on(monkeypatch):
    made, current = [], [0]

    @contextlib.contextmanager
    def on(stream):
        current.append(current[-1] if stream is None else stream.cuda_stream)
        yield
        current.pop()

    x, cache = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(3, 16, 4, 64, dtype=torch.float16)
    ints, freq, table = torch.zeros(2, dtype=torch.int32), torch.zeros(32), torch.zeros(2, 1, dtype=torch.int32)
    empty = torch.empty

    class Workspace:
        is_cuda, dtype = True, torch.uint8
        is_contiguous, data_ptr, numel = (lambda self: True), (lambda self: 1 << 40), (lambda self: 64)

    monkeypatch.setattr(kaio, "lib", Library)
    monkeypatch.setattr(kaio, "_host", lambda: False)
    monkeypatch.setattr(kaio, "_host_module", False)
    monkeypatch.setattr(kaio, "_strides", lambda t, *a: t.stride())
    monkeypatch.setattr(kaio, "_current_raw_stream", lambda device: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(current[-1]) or empty(*a, **kw))
    for stream, want in ((None, 0), (Stream(77), 77)):
        kaio.rope(x, ints, freq, stream=stream)
        kaio.rope_append(x, x, x, ints, freq, cache, cache.clone(), ints, stream=stream)
        kaio.paged_attention(x, cache, cache, table, ints, workspace=Workspace(), return_lse=True, stream=stream)
        assert made == [want] * 4
        made.clear()


@pytest.mark.gpu
@pytest.mark.parametrize("by_host", [True, False])
def test_do_not_meet_work_of_the_current_stream(monkeypatch, by_host):
    """The current stream has writes under way to memory of the results' sizes that was freed
    already, and reuses what is freed after the call at once."""
    from test_gpu_paged_attention import Problem
    if by_host and not kaio._host():
        pytest.skip("built without Python's or torch's headers")
    if not by_host:
        monkeypatch.setattr(kaio, "_host", lambda: False)
        monkeypatch.setattr(kaio, "_host_module", False)
    p = Problem([(64, 300)], 8, 2, 64)
    ws = kaio.paged_attention_workspace()
    pos, freq = torch.arange(64, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    side = torch.cuda.Stream()
    calls = [lambda **kw: (kaio.rope(p.q, pos, freq, **kw),), lambda **kw: p.run(workspace=ws, **kw)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        for _ in range(3):
            later = [torch.empty_like(w) for w in want]
            torch.cuda._sleep(20_000_000)
            for t in later:
                t.fill_(7.0)
            del later, t
            got = call(stream=side)
            side.synchronize()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            side.wait_stream(torch.cuda.current_stream())
            del got


@pytest.mark.gpu
def test_other_stream_objects_and_the_default_stream():
    q = torch.randn(5, 4, 64, device="cuda").half()
    pos, freq = torch.arange(5, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    want = kaio.rope(q, pos, freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (Stream(side.cuda_stream), Stream(0), torch.cuda.default_stream(), torch.cuda.current_stream(),
                   torch.cuda.ExternalStream(side.cuda_stream)):
        got = kaio.rope(q, pos, freq, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
