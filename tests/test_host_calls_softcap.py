"""The one-step host path takes a cap that is a whole number, as Python's own path does."""
import pytest
import torch

from qkv_projection_gb300 import kaio
from test_host_calls import host, same, tensors  # noqa: F401


@pytest.mark.gpu
def test_whole_caps_are_taken(host):  # noqa: F811
    a = tensors("cuda", t=6)
    ws = kaio.paged_attention_workspace()

    def attend(softcap):
        return host.paged_attention_scored(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["starts"], 4, None, True, 0, 0, ws,
                                           None, True, None, None, softcap, None, None, None)

    want = attend(3.0)
    assert want is not None
    same(attend(3), want)
    same(attend(True), attend(1.0))
    same(attend(0), attend(0.0))
    for other in (None, "3", 1 << 2000, -1, 300, 1e-50, torch.tensor(3.0)):
        assert attend(other) is None
