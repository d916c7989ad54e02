"""Written tensors whose rows share elements are refused, whatever the order of their
dimensions; padded and permuted ones are taken (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import paged_args, passes_validation, refused, rope_args

SHARED = [(64, 64), (256, 256), (128, 64), (200, 64), (64, 128), (128, 512), (320, 160)]     # token, head: 5 x 4 of 64
APART = [(256, 64), (512, 128), (64, 320), (72, 360), (264, 64), (288, 72)]


@pytest.mark.parametrize("ts,hs", SHARED)
def test_results_that_share_elements(ts, hs):
    for fn, args in ((kaio.lib().kaio_rope, rope_args), (kaio.lib().kaio_rope_append, rope_args)):
        refused(fn, args(o_ts=ts, o_hs=hs), "q_out: rows of a written tensor share elements")
    refused(kaio.lib().kaio_paged_attention, paged_args(o_ts=ts, o_hs=hs), "out: rows of a written tensor share elements")


@pytest.mark.parametrize("ts,hs", APART)
def test_results_that_do_not(ts, hs):
    passes_validation(kaio.lib().kaio_rope, rope_args(o_ts=ts, o_hs=hs))
    passes_validation(kaio.lib().kaio_paged_attention, paged_args(o_ts=ts, o_hs=hs))


def test_one_token_or_one_head_needs_no_stride():
    passes_validation(kaio.lib().kaio_rope, rope_args(tokens=1, o_ts=0, pos_stride=1))
    passes_validation(kaio.lib().kaio_rope, rope_args(heads=1, o_ts=64, o_hs=0))
    refused(kaio.lib().kaio_rope, rope_args(heads=1, o_ts=56, o_hs=0), "below dim")


@pytest.mark.parametrize("ps,ss,hs,ok", [
    (2048, 128, 64, True), (2048, 64, 1024, True), (4096, 128, 64, True), (128, 384, 64, True), (64, 384, 192, True),
    (2048, 128, 128, False), (1024, 128, 64, False), (128, 128, 64, False), (2048, 64, 64, False), (64, 128, 2048, False),
])
def test_caches(ps, ss, hs, ok):
    """3 pages of 16 slots of 2 heads of 64"""
    for name in "kv":
        args = rope_args(**{f"{name}c_ps": ps, f"{name}c_ss": ss, f"{name}c_hs": hs})
        if ok:
            passes_validation(kaio.lib().kaio_rope_append, args)
        else:
            refused(kaio.lib().kaio_rope_append, args, f"{name}_cache: rows of a written tensor share elements")
    # attention only reads the caches
    passes_validation(kaio.lib().kaio_paged_attention, paged_args(k_ps=ps, k_ss=ss, k_hs=hs))
