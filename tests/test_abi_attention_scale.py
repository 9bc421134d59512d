"""Scales that fp32 does not hold as a power of two's: refused on the host."""

import pytest

from test_abi_block import INVALID, change, refuse
from test_abi_cache import ATTEND


@pytest.mark.parametrize("scale", [3.4028234663852886e38, 2.4e38, 1e39])
def test_scales_that_overflow(q4lib, scale):
    """scores are in powers of two: scale log2(e) has to be a number"""
    refuse(q4lib, "q4_attention", change(ATTEND, _6=scale), INVALID)
