"""One token of very many heads: refused where the kernel's 32-bit count of its units would
not hold them (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import passes_validation, refused, rope_args


def one_token(**kw):
    return rope_args(**{**dict(tokens=1, axes=1, s0=kw["pairs"], s1=0, q_hs=kw["dim"], o_hs=kw["dim"], k_hs=kw["dim"],
                               v_hs=kw["dim"], kc_hs=kw["dim"], vc_hs=kw["dim"]), **kw})


@pytest.mark.parametrize("kw,ok", [
    (dict(heads=1 << 27, dim=256, pairs=128), False), (dict(heads=1 << 28, dim=256, pairs=128), False),   # 2^31, 2^32 units
    (dict(heads=1 << 27, dim=256, pairs=128, interleaved=1), False), (dict(heads=1 << 26, dim=256, pairs=8), False),
    (dict(heads=(1 << 26) - 1, dim=256, pairs=128), True),
    (dict(heads=1 << 27, dim=256, pairs=127), True),                                                      # a row a unit
])
def test_units_of_one_token(kw, ok):
    if ok:
        passes_validation(kaio.lib().kaio_rope, one_token(**kw))
    else:
        refused(kaio.lib().kaio_rope, one_token(**kw), "pieces of 16")


def test_units_with_the_cache():
    for kv_heads, ok in (((1 << 24), True), (1 << 25, False)):
        args = one_token(heads=(1 << 25) - 4, kv_heads=kv_heads, dim=256, pairs=128, page_size=1, num_pages=1)
        if ok:
            passes_validation(kaio.lib().kaio_rope_append, args)
        else:
            refused(kaio.lib().kaio_rope_append, args, "pieces of 16")
