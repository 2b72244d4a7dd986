"""CPU check of the attention's scale: it is held times log2 e, which has to be finite too."""

import math

import pytest

from test_abi_kv import attention, lib  # noqa: F401


@pytest.mark.parametrize("scale", [3e38, -3e38, math.inf, -math.inf, math.nan])
def test_scales_beyond_fp32_are_refused(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale) == -1


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 0.0, 1e-45])
def test_scales_within_fp32_pass_the_checks(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale, T=0) == 0
