"""A cap that is zero in 32 bits alone is refused, not left out (no GPU)."""
import pytest
import torch

from qkv_projection_gb300 import kaio


@pytest.mark.parametrize("softcap", [1e-50, -1e-50, 7e-46, 5e-324])
def test_caps_that_are_zero_in_32_bits(softcap):
    q, cache, i = torch.zeros(1, 2, 64).half(), torch.zeros(1, 16, 2, 64).half(), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="softcap"):
        kaio.paged_attention(q, cache, cache, i[None], i, softcap=softcap)


@pytest.mark.gpu
def test_caps_that_are_zero_in_32_bits_on_the_gpu():
    q, cache, i = torch.zeros(1, 2, 64).half().cuda(), torch.zeros(1, 16, 2, 64).half().cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    ws = kaio.paged_attention_workspace()
    for softcap in (1e-50, 7e-46):
        with pytest.raises(ValueError, match="softcap"):
            kaio.paged_attention(q, cache, cache, i[None], i, softcap=softcap, workspace=ws)
