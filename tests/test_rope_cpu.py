"""gw_rope_rows and gw_rope_cs_scaled: what the host refuses before any launch
(no GPU needed)."""

import ctypes

import pytest
import torch

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")


def _at(n=1 << 24):
    return ctypes.c_void_p(n)


def _rows(x=1 << 24, xr=1024, xh=256, y=1 << 28, yr=1024, yh=256, elem=0, rows=8, heads=4, dim=256, rot=256, pairs=0,
          pos=1 << 22, cs=1 << 22, max_pos=100, status=None):
    return gw.lib().gw_rope_rows(_at(x), xr, xh, _at(y), yr, yh, elem, rows, heads, dim, rot, pairs, 0, _at(pos),
                                 _at(cs), max_pos, _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(elem=3), dict(elem=-1), dict(pairs=2), dict(rows=-1), dict(heads=-1),
    dict(dim=1, rot=1), dict(dim=1025, rot=256), dict(rot=0), dict(rot=255), dict(rot=258), dict(max_pos=0),
    dict(x=0), dict(y=0), dict(x=(1 << 24) + 1), dict(y=(1 << 28) + 2, elem=2), dict(pos=0), dict(pos=(1 << 22) + 2),
    dict(cs=0), dict(cs=(1 << 22) + 8), dict(status=(1 << 22) + 2),
    dict(xr=-1024), dict(yh=-256), dict(xr=(1 << 40) + 1),
    dict(yh=255), dict(yr=1023), dict(yr=0), dict(yh=0),                      # rows of y overlap
    dict(yr=256, yh=8 * 256 - 1),                                             # head-major, one element short
    dict(y=1 << 24, yr=2048), dict(y=1 << 24, xh=512, xr=2048, yr=2048),      # in place, other strides
    dict(y=(1 << 24) + 2), dict(y=(1 << 24) + 2 * (8 * 1024 - 1)),            # x and y overlap
    dict(x=(1 << 28) + 2 * (8 * 1024 - 1)),
])
def test_rope_rows_refuses(bad):
    assert _rows(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_rope_rows:")


def test_rope_rows_without_rows_does_nothing():
    assert _rows(rows=0, x=0, y=0, pos=0, cs=0) == gw.GW_OK
    assert _rows(heads=0) == gw.GW_OK


def _table(cs=1 << 24, theta=1e4, rot=128, dim=512, max_pos=10, scaling=True, **kw):
    f = dict(kind=0, reserved=0, factor=2.0, low=1.0, high=32.0, orig_max_pos=8192.0, amplitude=1.0)
    f.update(kw)
    sc = gw.RopeScaling(**f)
    return gw.lib().gw_rope_cs_scaled(_at(cs), theta, rot, dim, max_pos, ctypes.byref(sc) if scaling else None, None)


@pytest.mark.parametrize("bad", [
    dict(cs=0), dict(cs=(1 << 24) + 8), dict(theta=0.0), dict(theta=float("inf")), dict(theta=float("nan")),
    dict(rot=0), dict(rot=127), dict(rot=514, dim=1024), dict(rot=256, dim=128), dict(max_pos=0), dict(scaling=False),
    dict(kind=4), dict(kind=-1), dict(reserved=1), dict(amplitude=0.0), dict(amplitude=float("inf")), dict(amplitude=1e-7), dict(theta=1e-200, rot=512),
    dict(kind=1, factor=0.0), dict(kind=1, factor=float("nan")), dict(kind=2, factor=-1.0), dict(kind=2, rot=2, dim=2),
    dict(kind=3, low=-1.0), dict(kind=3, low=32.0), dict(kind=3, high=float("inf")), dict(kind=3, orig_max_pos=0.0),
    dict(kind=1, factor=5e-324),                                              # a frequency overflows
])
def test_rope_cs_scaled_refuses(bad):
    assert _table(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_rope_cs_scaled:")


def test_binding_refuses():
    x = torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(gw.GwError, match="not on a CUDA device"):
        gw.rope_rows(x, torch.zeros(4, dtype=torch.int32), torch.zeros(8, 4, 2))
    with pytest.raises(gw.GwError, match="unknown kind"):
        gw.rope_cs_scaled(1e4, 128, 512, 16, kind="cubic")
    with pytest.raises(gw.GwError, match="not on a CUDA device"):
        gw.rope_cs_scaled(1e4, 128, 512, 16, out=torch.zeros(16, 64, 2))
    with pytest.raises(gw.GwError, match="budget|CUDA"):
        gw.kv_evict_select(torch.zeros(1, 4), torch.zeros(1, dtype=torch.int32), 2, torch.zeros(1, 4, dtype=torch.int32),
                           torch.zeros(1, dtype=torch.int32))
