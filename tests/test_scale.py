"""sm_scale as the Python entry points take it (no GPU needed)."""
import math

import pytest

from bwd_sparse_mqa_gb300 import api


@pytest.mark.parametrize("value", [1e39, 1e300, 1e-46, 1e-300, 0.0, -1.0, math.inf, math.nan])
def test_scales_that_fp32_does_not_hold_are_refused(value):
    """The C ABI takes a float, of which 0 and what is not finite select D^-1/2."""
    with pytest.raises(ValueError):
        api._scale(value, 64)


@pytest.mark.parametrize("value", [1.0, 1e-44, 1e-30, 1e38, 0.125])
def test_scales_in_range_are_used_as_given(value):
    assert api._scale(value, 64) == value
    assert api._scale(None, 64) == 0.125
