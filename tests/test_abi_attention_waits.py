"""Refusals of the test entry that limits the waits of attention's kernel for chunks (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import BF16, CUDA_ERR, F16, UNSUPPORTED, paged_args, refused


def test_wait_limit_is_for_one_kernel():
    fn = lambda args, stream: kaio.lib().kaio_debug_paged_attention_wait_limit(args, 0, stream)   # noqa: E731
    wide = dict(dtype=F16, dim=72, max_new=9, q_ts=288, q_hs=72, o_ts=288, o_hs=72, k_ps=2304, k_ss=144, k_hs=72,
                v_ps=2304, v_ss=144, v_hs=72)
    for kw in (dict(dtype=BF16), dict(dim=64), dict(max_new=8), dict(num_pages=0), dict(max_pages=0)):
        refused(fn, paged_args(**{**wide, **kw}), "wait limit")
    refused(fn, paged_args(**{**wide, "window": -1}), "window")
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: made-up pointers go no further than the argument checks")
    assert fn(paged_args(**wide), None) in (CUDA_ERR, UNSUPPORTED)
