"""Bounded waits of the kernel for chunks, on the GPU: with a limit of nothing or of a few
microseconds waits give up at the start or anywhere in the pipeline. The host then reads
a timeout, the context stays usable, and so does the workspace: the counters of split
items are zero again, and the next regular call on it gives what it gave before."""
import pytest

from qkv_projection_gb300 import kaio
from test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu

COUNTERS = 4096      # bytes


@pytest.fixture
def limited(monkeypatch):
    """limited(p, ns, **kw): p.run(**kw) with waits limited to ns."""
    def run(p, ns, **kw):
        L = kaio.lib()
        with monkeypatch.context() as m:
            m.setattr(kaio, "_host", lambda: False)
            m.setattr(kaio, "_host_module", False)
            m.setattr(L, "kaio_paged_attention",
                      lambda args, stream: L.kaio_debug_paged_attention_wait_limit(args, ns, stream))
            return p.run(**kw)
    return run


@pytest.mark.parametrize("lens,heads,kv_heads,mask", [
    ([(100, 9000)], 8, 2, {}),                                                # one item over many CTAs
    ([(64, 5000), (3, 900), (300, 2000), (1, 4000)], 8, 2, dict(window=1500, sinks=5)),
    ([(40, 2000 + 100 * i) for i in range(30)], 16, 4, {}),                   # two split items in most shares
])
def test_a_timeout_spoils_neither_context_nor_workspace(limited, lens, heads, kv_heads, mask):
    p = Problem(lens, heads, kv_heads, 128, 32, seed=1)
    ws = kaio.paged_attention_workspace()
    kaio.device_status()
    want = p.run(workspace=ws, **mask)
    statuses = set()
    for ns in (0, 500, 1000, 1500, 2000, 3000, 5000, 0):
        limited(p, ns, workspace=ws, **mask)
        status = kaio.lib().kaio_device_status()
        assert status == kaio.KAIO_ERR_DEVICE_TIMEOUT or (ns and status == kaio.KAIO_OK)
        statuses.add(status)
        assert kaio.lib().kaio_device_status() == kaio.KAIO_OK               # the read cleared it
        assert not ws[:COUNTERS].any()
        got = p.run(workspace=ws, **mask)
        assert all((a == b).all() for a, b in zip(got, want))
    assert kaio.KAIO_ERR_DEVICE_TIMEOUT in statuses
    got = limited(p, 2_000_000_000, workspace=ws, **mask)
    assert all((a == b).all() for a, b in zip(got, want))
    assert kaio.lib().kaio_device_status() == kaio.KAIO_OK
