"""gw_tree_attn_global refuses out = q before any launch (no GPU needed)."""

import ctypes

import pytest

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")

M = 1 << 20


@pytest.mark.parametrize("layout,dtype", [(gw.LAYOUT_GLOBAL_FOLDED, gw.KV_BF16), (gw.LAYOUT_GLOBAL_FULL, gw.KV_BF16),
                                          (gw.LAYOUT_GLOBAL_FOLDED_E4M3, gw.KV_E4M3)])
@pytest.mark.parametrize("heads,rows", [(8, 4), (32, 64)])
def test_refused(layout, dtype, heads, rows):
    d, p = gw.PoolDesc(layout, dtype, M, 100, 16, 1, 512, 128), ctypes.c_void_p(256 * M)
    code = gw.lib().gw_tree_attn_global(ctypes.byref(d), p, p, heads, 2, p, p, p, 64, p, rows, 0.04, p, 1 << 32, None, None)
    assert code == gw.GW_ERR_INVALID_ARG and "out is q" in gw.last_error()
