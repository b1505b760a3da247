"""The workspace of gw_tree_attn_* holds every call of at most its size (no GPU needed)."""

import ctypes
import re

import pytest

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")

M = 1 << 20
GLOBAL = [(gw.LAYOUT_GLOBAL_FOLDED, gw.KV_BF16), (gw.LAYOUT_GLOBAL_FULL, gw.KV_BF16),
          (gw.LAYOUT_GLOBAL_FOLDED_E4M3, gw.KV_E4M3)]


def desc(layout, dtype, kvh=1):
    local = layout == gw.LAYOUT_LOCAL
    return gw.PoolDesc(layout, dtype, M, 100, 16, kvh, 256 if local else 512, 256 if local else 128)


def size(d, heads, batch, pages, rows, window=0):
    return gw.lib().gw_tree_workspace_bytes(ctypes.byref(d), heads, batch, pages, rows, window)


def need(d, heads, batch, pages, rows, window=0):
    """What a call asks for, by its refusal of a workspace of no bytes."""
    p = ctypes.c_void_p(256 * M)
    if d.layout == gw.LAYOUT_LOCAL:
        code = gw.lib().gw_tree_attn_local(ctypes.byref(d), p, p, heads, batch, p, p, p, pages, p, p, rows, window, 0.1, p,
                                           0, None, None)
    else:
        code = gw.lib().gw_tree_attn_global(ctypes.byref(d), p, p, heads, batch, p, p, p, pages, p, rows, 0.1, p, 0, None,
                                            None)
    assert code == gw.GW_ERR_WORKSPACE
    return int(re.search(r"< (\d+) needed", gw.last_error()).group(1))


@pytest.mark.parametrize("layout,dtype", GLOBAL)
@pytest.mark.parametrize("heads", [8, 16, 32])
@pytest.mark.parametrize("pages", [1, 4, 31, 64, 160, 1024, 8192])
def test_global_holds_smaller_calls(layout, dtype, heads, pages):
    d = desc(layout, dtype)
    before = 0
    for rows in range(1, 65):
        have = size(d, heads, 3, pages, rows)
        assert have >= before  # never less for more rows
        before = have
        for h in (8, 16, 32):
            for r in {1, 2, 4, 8, rows, max(1, rows // 2), max(1, rows - 1)}:
                if h <= heads and r <= rows:
                    for b, p in ((3, pages), (1, pages), (3, max(1, pages // 2)), (2, max(1, pages - 1))):
                        assert need(d, h, b, p, r) <= have, (h, b, p, r, rows)
        assert size(d, heads, 4, pages, rows) >= have and size(d, heads, 3, pages + 1, rows) >= have


@pytest.mark.parametrize("kvh,heads", [(4, 4), (4, 8), (2, 16), (1, 8)])
@pytest.mark.parametrize("window", [1, 64, 1024, 1 << 30])
@pytest.mark.parametrize("pages", [1, 31, 160, 4096])
def test_local_holds_smaller_calls(kvh, heads, window, pages):
    for dtype in (gw.KV_BF16, gw.KV_E4M3):
        d = desc(gw.LAYOUT_LOCAL, dtype, kvh)
        before = 0
        for rows in (1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 63, 64):
            have = size(d, heads, 3, pages, rows, window)
            assert have >= before
            before = have
            for h in (kvh, 2 * kvh, 4 * kvh, 8 * kvh):
                for r in {1, 4, 16, rows, max(1, rows // 2), max(1, rows - 1)}:
                    if h <= heads and r <= rows:
                        for b, p, w in ((3, pages, window), (1, pages, window), (3, max(1, pages // 2), window),
                                        (3, pages, max(1, window // 2)), (3, pages, max(1, window - 1))):
                            assert need(d, h, b, p, r, w) <= have, (h, b, p, r, w, rows)


def test_the_default_bound_holds_a_small_step():
    """64 rows over 2560 tokens have one chunk, 4 rows five."""
    for layout, dtype in GLOBAL:
        d = desc(layout, dtype)
        assert size(d, 8, 4, 160, 64) >= need(d, 8, 4, 160, 4) > 1 << 20


@pytest.mark.parametrize("layout,dtype", GLOBAL)
def test_a_lone_sequence_is_cut(layout, dtype):
    """2560 tokens, 16 drafts of 32 heads: three chunks of four blocks, two halves each, whose parts are 128 KB."""
    assert need(desc(layout, dtype), 32, 1, 160, 16) >= 3 * 4 * 2 << 17
