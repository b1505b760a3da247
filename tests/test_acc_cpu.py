"""gw_decode_attn_global_acc: what the host refuses before any launch (no GPU
needed), and its workspace size."""

import ctypes

import pytest

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")


def _at(n=1 << 24):
    return ctypes.c_void_p(n)


def _desc(layout=gw.LAYOUT_GLOBAL_FOLDED, dtype=gw.KV_BF16, base=1 << 20):
    local = layout == gw.LAYOUT_LOCAL
    return gw.PoolDesc(layout, dtype, base, 100, 16, 4 if local else 1, 256 if local else 512, 256 if local else 128)


def _call(desc=None, q=1 << 24, out=1 << 24, lse=1 << 24, acc=1 << 24, stride=1024, decay=1.0, hq=32, batch=2, pages=64,
          scale=0.04, ws=1 << 28, ws_bytes=1 << 30, status=0):
    f = _at()
    return gw.lib().gw_decode_attn_global_acc(ctypes.byref(desc or _desc()), _at(q), _at(out), _at(lse), _at(acc),
                                              stride, decay, hq, batch, f, f, f, pages, scale, _at(ws), ws_bytes,
                                              _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(acc=0), dict(acc=(1 << 24) + 2), dict(lse=(1 << 24) + 1), dict(stride=1023), dict(stride=-1),
    dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf")), dict(q=0), dict(out=(1 << 24) + 8),
    dict(pages=0), dict(pages=1 << 27, stride=1 << 40), dict(scale=0.0), dict(ws=0), dict(batch=-1),
    dict(desc=_desc(gw.LAYOUT_LOCAL)), dict(status=(1 << 24) + 1),
])
def test_refuses(bad):
    assert _call(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_decode_attn_global_acc:")


def test_unsupported_and_workspace():
    assert _call(hq=12) == gw.GW_ERR_UNSUPPORTED
    assert _call(batch=4097) == gw.GW_ERR_UNSUPPORTED
    assert _call(desc=_desc(dtype=gw.KV_E4M3)) == gw.GW_ERR_UNSUPPORTED
    assert _call(batch=0) == gw.GW_OK
    for layout, dtype in ((gw.LAYOUT_GLOBAL_FOLDED, gw.KV_BF16), (gw.LAYOUT_GLOBAL_FULL, gw.KV_BF16),
                          (gw.LAYOUT_GLOBAL_FOLDED_E4M3, gw.KV_E4M3)):
        d = _desc(layout, dtype, base=0)
        need = gw.lib().gw_attn_acc_workspace_bytes(ctypes.byref(d), 32, 2, 64)
        plain = gw.lib().gw_attn_workspace_bytes(ctypes.byref(d), 32, 2, 1024, 1, 0)
        assert need >= plain + 2 * 1024 * 32 * 4
        assert _call(desc=_desc(layout, dtype), ws_bytes=need - 1) == gw.GW_ERR_WORKSPACE
        assert str(need) in gw.last_error()


def test_workspace_bytes_refuses():
    size = gw.lib().gw_attn_acc_workspace_bytes
    d = _desc()
    assert size(ctypes.byref(_desc(gw.LAYOUT_LOCAL)), 32, 2, 64) == 0
    assert gw.last_error().startswith("gw_attn_acc_workspace_bytes:")
    assert size(ctypes.byref(d), 0, 2, 64) == 0 and size(ctypes.byref(d), 32, -1, 64) == 0
    assert size(ctypes.byref(d), 32, 2, 0) == 0 and size(ctypes.byref(d), 32, 2, 1 << 27) == 0
    # long contexts in many slots: sizes past 32 bits
    assert size(ctypes.byref(d), 32, 256, 8192) > 256 * 131072 * 32 * 4
