"""Limits of the 4-bit cache's calls that no launch is needed for."""
import pytest

import post_weight_quantization_21_amd as gq
from test_kv_abi import INV, attention, cache


@pytest.mark.parametrize("scale", [1.71e38, 3.39e38, float("inf")])
def test_scales_that_overflow_are_refused(scale):
    """The scores are taken in log2: a scale is multiplied by log2 e, which passes fp32's end above 2^127.9."""
    assert attention(cache(), scale=scale) == INV
    assert b"scale" in gq.load_library().gptq_last_error()


def test_largest_scale_passes():
    assert attention(cache(), scale=2.0 ** 127, n_seq=0, Q=None, O=None, table=None, lens=None, ws=None, ws_bytes=0) == gq.OK
