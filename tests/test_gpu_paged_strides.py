"""Attention over caches in strides of their own: heads or pages that are one memory
(expanded), pages inside slots, and padding of every dimension. The tolerance is that of
test_gpu_paged_attention.py; what the views hold is all that matters."""
import pytest

from test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu


def views(p, how):
    """k and v of p, in place of its own."""
    import torch
    pages, page, kh, d = p.kc.shape
    out = []
    for c in (p.kc, p.vc):
        if how == "one head":
            v = c[:, :, :1].expand(pages, page, kh, d)
        elif how == "one page":
            v = c[:1].expand(pages, page, kh, d)
        elif how == "pages inside slots":
            v = c.transpose(0, 1).contiguous().transpose(0, 1)
        elif how == "pages innermost":
            v = c.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
        else:
            v = torch.full((pages + 1, page + 3, kh + 2, d + 24), float("nan"), dtype=c.dtype, device="cuda")
            v = v[:pages, 2:page + 2, 1:kh + 1, 8:d + 8]
            v.copy_(c)
        out.append(v)
    p.kc, p.vc = out


@pytest.mark.parametrize("how", ["one head", "one page", "pages inside slots", "pages innermost", "padded"])
@pytest.mark.parametrize("lens", [[(1, 700), (1, 33)], [(150, 700), (3, 40)]])
@pytest.mark.parametrize("d,dtype", [(128, "float16"), (64, "bfloat16"), (72, "float16")])
def test_caches_in_strides_of_their_own(lens, how, d, dtype):
    p = Problem(lens, 6, 3, d, 32, dtype, seed=d)
    views(p, how)
    p.verify()
    p.verify(window=90, sinks=5)
