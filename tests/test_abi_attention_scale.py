"""The scale is held times log2(e): one that is finite only by itself is refused (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import paged_args, passes_validation, refused


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 2.99e38])
def test_scale_times_log2_e_is_finite(scale):
    refused(kaio.lib().kaio_paged_attention, paged_args(scale=scale), "scale")


def test_scales_taken():
    for scale in (0.0, -0.3, 2.3e38, -2.3e38, 1e-45):
        passes_validation(kaio.lib().kaio_paged_attention, paged_args(scale=scale))
