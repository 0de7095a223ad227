"""Caps whose squares leave fp32's range are refused by the calls that take one, on the CPU."""
import pytest

from tests.test_paged_range_refusals import attend, range_call


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("scale, cap, code", [
    (0.01, 9e-19, 2), (1e-4, 1e-20, 2), (1e-30, 1e-38, 2), (100.0, 1.1e18, 2), (1e10, 1e25, 2),
    (0.01, 1.1e-18, 9), (1e-4, 1e-10, 9), (100.0, 9e17, 9), (0.1, 0.0, 9)])  # 9: only the workspace is too small
def test_caps(lib, scale, cap, code, dtype):
    assert attend(lib, dtype=dtype, scale=scale, cap=cap, n=8) == code
    for back in (False, True):
        assert range_call(lib, back, dtype=dtype, scale=scale, cap=cap, n=8) == code
