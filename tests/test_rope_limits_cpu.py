"""gw_rope_rows and gw_rope_cs_scaled: refusals at the ends of their ranges (no
GPU needed)."""

import pytest

from tests.test_rope_cpu import _rows, _table, gw


@pytest.mark.parametrize("heads", [(1 << 30) + 1, 2 ** 31 - 1])
def test_more_heads_than_are_counted(heads):
    assert _rows(rows=1, heads=heads, dim=2, rot=2, xh=2, yh=2, x=1 << 24, y=1 << 40) == gw.GW_ERR_INVALID_ARG
    assert "2^30" in gw.last_error()


@pytest.mark.parametrize("theta,factor", [(1e300, 1e20), (1e-300, 1e-20), (1e-200, 1e-109)])
def test_an_ntk_base_outside_float64(theta, factor):
    """An infinite base has no frequencies but 1 and 0, a subnormal one has lost
    its bits."""
    assert _table(theta=theta, kind=2, factor=factor, rot=2) == gw.GW_ERR_INVALID_ARG
    assert "range" in gw.last_error()
