"""The one-step host path of the cache's upkeep and of the scored attention against the code in
Python: it leaves to Python whatever it does not take, and gives the same results."""
import pytest
import torch

from qkv_projection_gb300 import kaio
from test_host_calls import both, host, same, tensors  # noqa: F401

I32 = torch.int32


def arguments(a):
    refs, table, lens = torch.zeros(9, dtype=I32), a["table"].cpu().clone(), a["lens"].cpu().clone()
    attend = (a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"], None, None, True, 0, 0,
              torch.zeros(64, dtype=torch.uint8), None, False, None, None, 30.0, None, None, None)
    return {"paged_attention_scored": attend, "cache_copy_pages": ([a["kc"], a["vc"]], lens, lens, None),
            "cache_fork": (refs, table, lens, lens, 16, None), "cache_truncate": (refs, table, lens, lens, 16, None),
            "cache_append": (refs, table, lens, None, 2, 16, None), "cache_compact": (refs, table, lens, 16, 3, None)}


def test_leaves_what_it_does_not_take(host):  # noqa: F811
    for name, args in arguments(tensors("cpu")).items():
        call = getattr(host, name)
        assert call(*args) is None                    # on the CPU
        assert call(*args[:-1]) is None               # too few
        assert call() is None
        for i in range(len(args)):
            for other in (None, 3, "x", object(), torch.zeros(2), float("nan"), 1 << 80, [], [1], (torch.zeros(2),) * 600):
                assert call(*args[:i], other, *args[i + 1:]) is None


def test_bind_more_takes_six_addresses(host):  # noqa: F811
    with pytest.raises(TypeError):
        host.bind_more(1)
    with pytest.raises(TypeError):
        host.bind_more("a", 2, 3, 4, 5, 6)


@pytest.mark.gpu
def test_scored_attention_the_same_either_way(host, monkeypatch):  # noqa: F811
    a = tensors("cuda", t=6)
    docs, prefix = (torch.tensor(v, dtype=I32, device="cuda") for v in ([0, 3, 0, 0, 5, 5], [7, 0]))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0], device="cuda")
    ws = kaio.paged_attention_workspace()
    for kw in (dict(softcap=3.0), dict(slopes=slopes), dict(prefix_lens=prefix, softcap=2), dict(doc_starts=docs),
               dict(softcap=3.0, slopes=slopes, prefix_lens=prefix, doc_starts=docs, window=4, sinks=1)):
        same(*both(monkeypatch, lambda: kaio.paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"],
                                                             max_new=4, return_lse=True, workspace=ws, **kw)))
    for error, match, kw in ((ValueError, "slopes", dict(slopes=slopes[:2])), (TypeError, "doc_starts", dict(doc_starts=docs.long())),
                             (kaio.KaioError, "softcap", dict(softcap=-1.0)), (TypeError, None, dict(softcap="x"))):
        for hold in (False, True):
            with monkeypatch.context() as m, pytest.raises(error, match=match):
                if hold:
                    m.setattr(kaio, "_host", lambda: False)
                    m.setattr(kaio, "_host_module", False)
                kaio.paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"], workspace=ws, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("given_stream", [False, True])
def test_upkeep_the_same_either_way(host, monkeypatch, given_stream):  # noqa: F811
    i = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    stream = torch.cuda.Stream() if given_stream else None

    def run():
        caches = [torch.arange(9 * 16 * 64, device="cuda").remainder(100).half().view(9, 16, 1, 64) * (k + 1) for k in range(3)]
        refs, table, lens, starts = i([1, 2, 0, 0, 1, 0, 0, 0, 1]), i([[0, 1, 7, 7], [4, 1, 8, 7]]), i([18, 40]), i([0, 20, 23])
        parents, kept = i([1, 1]), i([100, 17])
        torch.cuda.synchronize()
        books = refs, table, lens
        made = kaio.cache_append(*books, starts, 23, 16, stream=stream)
        kaio.cache_copy_pages(tuple(caches), made[1], made[2], stream=stream)
        kaio.cache_fork(*books, parents, 16, stream=stream)
        made += kaio.cache_append(*books, None, 2, 16, stream=stream)
        kaio.cache_truncate(*books, kept, 16, stream=stream)
        made += kaio.cache_compact(*books, 16, 5, stream=stream)
        torch.cuda.synchronize()
        return (*made, *books, *caches)

    same(*both(monkeypatch, run))
