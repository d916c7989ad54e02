"""Rotation in place with the cache write: k and v may lie beside q in one packed buffer,
but not on q's own elements (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import passes_validation, ptr, refused, rope_args


def packed(order="qkv", **kw):
    """q [5, 4, 64] in place, k and v [5, 2, 64], the parts of rows of 512 values."""
    at = {"qkv": (0, 256, 384), "kvq": (256, 0, 128), "kqv": (128, 0, 384)}[order]
    a = dict(q=ptr(0, 2 * at[0]), q_out=ptr(0, 2 * at[0]), k=ptr(0, 2 * at[1]), v=ptr(0, 2 * at[2]), q_ts=512, o_ts=512,
             k_ts=512, v_ts=512)
    return rope_args(**{**a, **kw})


@pytest.mark.parametrize("order", ["qkv", "kvq", "kqv"])
def test_parts_of_one_buffer(order):
    passes_validation(kaio.lib().kaio_rope_append, packed(order))


def test_heads_outside_tokens():
    # [8 heads, 5 tokens, 64]: q the first four, k and v two each
    passes_validation(kaio.lib().kaio_rope_append, rope_args(
        q=ptr(0), q_out=ptr(0), k=ptr(0, 2 * 4 * 320), v=ptr(0, 2 * 6 * 320), q_ts=64, o_ts=64, k_ts=64, v_ts=64,
        q_hs=320, o_hs=320, k_hs=320, v_hs=320))


@pytest.mark.parametrize("kw,name", [
    (dict(k=ptr(0)), "k"), (dict(v=ptr(0)), "v"),                          # k or v is q
    (dict(k=ptr(0, 2 * 192)), "k"),                                        # k begins in q's last head
    (dict(v=ptr(0, 2 * 448)), "v"),                                        # v runs into the next token's q
    (dict(k=ptr(0, -2 * 64)), "k"),                                        # and k from before the first
    (dict(v=ptr(0, 2 * (2 * 512 + 64))), "v"),                             # two tokens on
    (dict(k_ts=256), "k"), (dict(v_ts=1024), "v"),                         # other strides
])
def test_shared_elements(kw, name):
    refused(kaio.lib().kaio_rope_append, packed(**kw), f"output q_out overlaps input {name}")


def test_one_token():
    one = dict(tokens=1, q=ptr(0), q_out=ptr(0), pos_stride=1, q_ts=0, o_ts=0, k_ts=0, v_ts=0)
    passes_validation(kaio.lib().kaio_rope_append, rope_args(**one, k=ptr(0, 512), v=ptr(0, 768)))
    refused(kaio.lib().kaio_rope_append, rope_args(**one, k=ptr(0, 384), v=ptr(0, 768)), "overlaps input k")
