"""gw_kv_evict_select and gw_kv_evict_compact: what the host refuses before
any launch (no GPU needed)."""

import ctypes

import pytest

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")


def _at(n=1 << 24):
    return ctypes.c_void_p(n)


def _select(acc=1 << 24, stride=1000, batch=4, lens=1 << 24, budget=100, sinks=4, recent=16, idx=1 << 25, idx_stride=100,
            n=1 << 26, status=0):
    return gw.lib().gw_kv_evict_select(_at(acc), stride, batch, _at(lens), budget, sinks, recent, _at(idx), idx_stride,
                                       _at(n), _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=65536), dict(budget=0), dict(budget=-1), dict(sinks=-1), dict(recent=-1),
    dict(sinks=90, recent=11), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(stride=0), dict(stride=(1 << 40) + 1),
    dict(idx_stride=99), dict(idx_stride=(1 << 40) + 1), dict(acc=0), dict(acc=(1 << 24) + 2), dict(lens=0),
    dict(lens=(1 << 24) + 1), dict(idx=0), dict(idx=(1 << 25) + 2), dict(n=0), dict(n=(1 << 26) + 3), dict(n=1 << 24),
    dict(status=(1 << 24) + 2),
])
def test_select_refuses(bad):
    assert _select(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_kv_evict_select:")


def _desc(layout=gw.LAYOUT_GLOBAL_FOLDED, dtype=gw.KV_BF16, base=1 << 20):
    local = layout == gw.LAYOUT_LOCAL
    return gw.PoolDesc(layout, dtype, base, 100, 16, 4 if local else 1, 256 if local else 512, 256 if local else 128)


def _compact(desc=None, batch=4, table=1 << 24, pages=64, lens=1 << 24, idx=1 << 25, idx_stride=100, n=1 << 26, dst=0,
             dst_pages=0, acc=1 << 27, stride=1024, status=0):
    return gw.lib().gw_kv_evict_compact(ctypes.byref(desc or _desc()), batch, _at(table), pages, _at(lens), _at(idx),
                                        idx_stride, _at(n), _at(dst) if dst else None, dst_pages,
                                        _at(acc) if acc else None, stride, _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(desc=_desc(base=0)), dict(desc=_desc(base=(1 << 20) + 16)), dict(batch=-1), dict(batch=65536), dict(table=0),
    dict(table=(1 << 24) + 2), dict(pages=0), dict(pages=1 << 27, stride=1 << 32), dict(lens=0), dict(idx=0),
    dict(idx=(1 << 25) + 2), dict(idx_stride=0), dict(n=0), dict(n=1 << 24), dict(dst=(1 << 24) + 2, dst_pages=4),
    dict(dst=1 << 23, dst_pages=0), dict(acc=(1 << 27) + 2), dict(stride=1023), dict(stride=(1 << 40) + 1),
    dict(status=(1 << 24) + 2),
])
def test_compact_refuses(bad):
    assert _compact(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_kv_evict_compact:")


def test_local_pools_and_empty_batches():
    assert _compact(desc=_desc(gw.LAYOUT_LOCAL)) == gw.GW_ERR_UNSUPPORTED
    assert "window" in gw.last_error()
    assert _compact(desc=_desc(dtype=gw.KV_E4M3)) == gw.GW_ERR_UNSUPPORTED
    assert _compact(batch=0, table=0, lens=0, idx=0, n=0) == gw.GW_OK
    assert _select(batch=0, acc=0, lens=0, idx=0, n=0) == gw.GW_OK
