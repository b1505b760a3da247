"""gw_rope_rows and gw_rope_cs_scaled: refusals at the ends of their ranges (no
GPU needed)."""

import pytest

from tests.test_rope_cpu import _rows, gw


@pytest.mark.parametrize("heads", [(1 << 30) + 1, 2 ** 31 - 1])
def test_more_heads_than_are_counted(heads):
    assert _rows(rows=1, heads=heads, dim=2, rot=2, xh=2, yh=2, x=1 << 24, y=1 << 40) == gw.GW_ERR_INVALID_ARG
    assert "2^30" in gw.last_error()
