"""The workspace that an attention call makes for itself belongs to the call's stream: it
is zeroed there, before the kernel, and the allocator reuses it there, after it."""
import contextlib

import pytest
import torch

from qkv_projection_gb300 import kaio


class Recorder:
    """Stands in for the library: a workspace of 64 bytes, and the stream of a launch."""

    def __init__(self):
        self.current, self.zeroed, self.launched = 0, [], []

    def kaio_paged_attention_workspace(self, n):
        n._obj.value = 64
        return kaio.KAIO_OK

    def kaio_paged_attention(self, args, stream):
        self.launched.append(stream)
        return kaio.KAIO_OK

    @contextlib.contextmanager
    def on(self, stream):
        before = self.current
        self.current = before if stream is None else stream.cuda_stream
        yield
        self.current = before


class Memory:
    """A tensor of which only a beginning is zeroed."""
    is_cuda, dtype = True, torch.uint8

    def __init__(self, recorder):
        self.recorder, self.made = recorder, recorder.current

    def __getitem__(self, part):
        assert part == slice(None, kaio.KAIO_PAGED_ATTENTION_COUNTERS)
        return self

    def zero_(self):
        assert self.made == self.recorder.current
        self.recorder.zeroed.append(self.made)

    is_contiguous, data_ptr, numel = (lambda self: True), (lambda self: 1 << 40), (lambda self: 64)


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


def test_is_zeroed_on_the_stream_that_the_kernel_runs_on(monkeypatch):
    r = Recorder()
    q, cache = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32)
    out = torch.empty_like(q)
    monkeypatch.setattr(kaio, "lib", lambda: r)
    monkeypatch.setattr(kaio, "_host", lambda: False)
    monkeypatch.setattr(kaio, "_host_module", False)
    monkeypatch.setattr(kaio, "_strides", lambda t, *a: t.stride())
    monkeypatch.setattr(kaio, "_current_raw_stream", lambda device: r.current)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", r.on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: Memory(r))
    for stream, want in ((None, 0), (Stream(77), 77), (Stream(5), 5)):
        kaio.paged_attention(q, cache, cache, table, lens, out=out, stream=stream)
        assert r.zeroed.pop() == want and r.launched.pop() == want
    with r.on(Stream(9)):
        kaio.paged_attention(q, cache, cache, table, lens, out=out)
    assert r.zeroed.pop() == 9 and r.launched.pop() == 9


@pytest.mark.gpu
def test_does_not_wait_for_or_meet_work_of_the_current_stream():
    """The current stream is busy, and what it allocates before and after the call is
    memory of the workspace's size full of ones."""
    from test_gpu_paged_attention import Problem
    for lens in ([(1, 9000)], [(64, 7000), (1, 3000)]):
        p = Problem(lens, 8, 2, 64, 64)
        ws = kaio.paged_attention_workspace()
        want = p.run(workspace=ws)
        size = ws.numel()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        del ws
        for _ in range(3):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(20_000_000)
            got = p.run(stream=side)
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            torch.cuda.synchronize()


def test_the_header_says_what_has_to_be_zero():
    assert f"#define KAIO_PAGED_ATTENTION_COUNTERS {kaio.KAIO_PAGED_ATTENTION_COUNTERS}\n" in open(kaio.HEADER).read()


@pytest.mark.gpu
def test_only_the_counters_are_zeroed_and_the_rest_may_hold_anything():
    from test_gpu_paged_attention import Problem
    size = kaio.paged_attention_workspace().numel()
    n = kaio.KAIO_PAGED_ATTENTION_COUNTERS
    dirty = torch.full((size,), 255, dtype=torch.uint8, device="cuda")       # as floats and as counters: NaN, all ones
    at = dirty.data_ptr()
    del dirty
    ws = kaio.paged_attention_workspace()
    assert ws.data_ptr() == at and not ws[:n].any() and (ws[n:] == 255).all()
    for lens in ([(1, 9000)], [(64, 7000), (1, 3000)], [(100, 300)]):
        p = Problem(lens, 8, 2, 128, 32)
        want = p.run(workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
        ws[n:] = 255
        assert all(torch.equal(a, b) for a, b in zip(p.run(workspace=ws), want))
