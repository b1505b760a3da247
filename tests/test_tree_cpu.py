"""gw_norm_rope_append, gw_tree_attn_*, gw_tree_accept and gw_kv_tree_move: what
the host refuses before any launch (no GPU needed), and the workspace sizes."""

import ctypes

import pytest

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")

M = 1 << 20


def _at(n=1 << 24):
    return ctypes.c_void_p(n)


def _desc(layout=gw.LAYOUT_LOCAL, dtype=gw.KV_BF16, base=M, kvh=4, pages=100):
    local = layout == gw.LAYOUT_LOCAL
    return gw.PoolDesc(layout, dtype, base, pages, 16, kvh if local else 1, 256 if local else 512, 256 if local else 128)


FOLDED, FULL, E4 = gw.LAYOUT_GLOBAL_FOLDED, gw.LAYOUT_GLOBAL_FULL, gw.LAYOUT_GLOBAL_FOLDED_E4M3


# ---- gw_norm_rope_append -------------------------------------------------------
def _norm(desc=None, q=32 * M, qr=2048, qh=256, k=64 * M, kr=1024, kh=256, v=96 * M, vr=1024, vh=256, rows=4, hq=8,
          qw=M, kw=M, eps=1e-6, v_norm=1, slot=M, pos=M, cs=M, max_pos=100, out=128 * M, status=0):
    return gw.lib().gw_norm_rope_append(ctypes.byref(desc or _desc()), _at(q), qr, qh, _at(k), kr, kh, _at(v), vr, vh,
                                        rows, hq, _at(qw), _at(kw), eps, v_norm, _at(slot), _at(pos), _at(cs), max_pos,
                                        _at(out), _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(desc=_desc(base=0)), dict(rows=-1), dict(hq=0), dict(hq=1025), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(max_pos=0), dict(q=0), dict(k=0), dict(v=0), dict(out=0),
    dict(q=32 * M + 8), dict(k=64 * M + 2), dict(v=96 * M + 8), dict(out=128 * M + 8), dict(qr=2044), dict(kh=257),
    dict(vr=-8), dict(kr=(1 << 40) + 8), dict(qw=0), dict(kw=M + 4), dict(slot=0), dict(pos=M + 2), dict(cs=M + 8),
    dict(status=M + 1),
    # out over part of q, over k, over v, and q in place with gaps
    dict(out=32 * M + 4096), dict(out=64 * M), dict(out=96 * M - 16), dict(out=32 * M, qr=2056),
    dict(out=32 * M, qh=264, qr=8 * 264),
    # folded pools: V is K's projection, normed
    dict(desc=_desc(FOLDED), qr=4096, qh=512), dict(desc=_desc(FOLDED), qr=4096, qh=512, v=64 * M, v_norm=0),
    dict(desc=_desc(FOLDED), qr=4096, qh=512, v=64 * M, vr=512), dict(desc=_desc(E4, gw.KV_E4M3), qr=4096, qh=512),
])
def test_norm_refuses(bad):
    assert _norm(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_norm_rope_append:")


def test_norm_unsupported_and_empty():
    assert _norm(desc=_desc(FULL, gw.KV_E4M3)) == gw.GW_ERR_UNSUPPORTED
    assert _norm(rows=0, q=0, k=0, v=0, out=0, slot=0, pos=0) == gw.GW_OK


# ---- gw_tree_attn_local / _global ------------------------------------------------
def _local(desc=None, q=M, out=M, hq=8, batch=2, cu=M, lens=M, table=M, pages=64, mask=M, pos=M, rows=16, window=32,
           scale=0.06, ws=256 * M, ws_bytes=1 << 32, status=0):
    return gw.lib().gw_tree_attn_local(ctypes.byref(desc or _desc()), _at(q), _at(out), hq, batch, _at(cu), _at(lens),
                                       _at(table), pages, _at(mask), _at(pos), rows, window, scale, _at(ws), ws_bytes,
                                       _at(status) if status else None, None)


def _global(desc=None, q=M, out=M, hq=8, batch=2, cu=M, lens=M, table=M, pages=64, mask=M, rows=16, scale=0.04,
            ws=256 * M, ws_bytes=1 << 32, status=0):
    return gw.lib().gw_tree_attn_global(ctypes.byref(desc or _desc(FOLDED)), _at(q), _at(out), hq, batch, _at(cu),
                                        _at(lens), _at(table), pages, _at(mask), rows, scale, _at(ws), ws_bytes,
                                        _at(status) if status else None, None)


COMMON = [dict(batch=-1), dict(q=0), dict(q=M + 8), dict(out=0), dict(out=M + 8), dict(cu=0), dict(cu=M + 2),
          dict(lens=0), dict(table=M + 1), dict(pages=0), dict(pages=1 << 26), dict(mask=0), dict(mask=M + 4),
          dict(rows=0), dict(rows=65), dict(rows=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
          dict(scale=float("nan")), dict(ws=0), dict(ws=256 * M + 128), dict(status=M + 2), dict(hq=0)]


@pytest.mark.parametrize("bad", COMMON + [dict(desc=_desc(FOLDED)), dict(desc=_desc(base=M + 16)), dict(pos=0),
                                          dict(pos=M + 1), dict(window=0), dict(window=-5), dict(hq=6)])
def test_local_refuses(bad):
    assert _local(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_tree_attn_local:")


@pytest.mark.parametrize("bad", COMMON + [dict(desc=_desc()), dict(desc=_desc(FULL, base=0))])
def test_global_refuses(bad):
    assert _global(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_tree_attn_global:")


def test_attn_unsupported_workspace_and_empty():
    assert _local(hq=12) == gw.GW_ERR_UNSUPPORTED and _local(hq=64) == gw.GW_ERR_UNSUPPORTED
    assert _global(hq=12) == gw.GW_ERR_UNSUPPORTED and _global(hq=64) == gw.GW_ERR_UNSUPPORTED
    assert _local(batch=257) == gw.GW_ERR_UNSUPPORTED and _global(batch=257) == gw.GW_ERR_UNSUPPORTED
    assert _global(desc=_desc(FOLDED, gw.KV_E4M3)) == gw.GW_ERR_UNSUPPORTED
    assert _local(batch=0, q=0, out=0, cu=0, mask=0, ws=0) == gw.GW_OK
    assert _global(batch=0, q=0, out=0, cu=0, mask=0, ws=0) == gw.GW_OK
    size = gw.lib().gw_tree_workspace_bytes
    need = size(ctypes.byref(_desc(base=0)), 8, 2, 64, 16, 1024)
    assert need > 0 and _local(window=1024, ws_bytes=need - 1) == gw.GW_ERR_WORKSPACE
    assert str(need) in gw.last_error()
    for layout, dtype in ((FOLDED, gw.KV_BF16), (FULL, gw.KV_BF16), (E4, gw.KV_E4M3)):
        need = size(ctypes.byref(_desc(layout, dtype, base=0)), 32, 2, 512, 16, 0)
        assert need > 0 and _global(desc=_desc(layout, dtype), hq=32, pages=512, ws_bytes=need - 1) == gw.GW_ERR_WORKSPACE


def _chunks(tiles, aim, most, blocks):
    chunks = min(-(-tiles // aim), most, max(1, 76 // blocks))
    return -(-tiles // -(-tiles // chunks))


@pytest.mark.parametrize("layout,heads,kvh,window", [
    (gw.LAYOUT_LOCAL, 8, 4, 1), (gw.LAYOUT_LOCAL, 8, 4, 65), (gw.LAYOUT_LOCAL, 32, 4, 1024),
    (gw.LAYOUT_LOCAL, 8, 8, 1 << 30), (FOLDED, 8, 1, 0), (FULL, 16, 1, 0), (FOLDED, 32, 1, 0)])
@pytest.mark.parametrize("pages,rows", [(1, 1), (5, 7), (64, 16), (1000, 64), (8192, 33)])
def test_workspace_holds_every_step(layout, heads, kvh, window, pages, rows):
    """No mix of rows and lengths up to the bounds needs more units than the workspace holds."""
    local = layout == gw.LAYOUT_LOCAL
    group, copies, aim, most = (heads // kvh, kvh, 18, 38) if local else (heads, 2, 40, 38)
    if not local and rows * heads <= 64:
        aim, most = 8, 76
    got = gw.lib().gw_tree_workspace_bytes(ctypes.byref(_desc(layout, kvh=kvh, base=0)), heads, 3, pages, rows, window)
    per = 128 // group
    cap = group * min(per, rows)
    worst = 0
    for n in range(1, rows + 1):
        blocks = -(-n // per)
        lens = {min(pages * 16, max(n, x)) for e in range(1, 18) for x in
                (n, (1 << e) - 1, 1 << e, (1 << e) + 1, 3 << e, window + n, window + n + 63, pages * 16)}
        for L in lens:
            if L < n:
                continue
            first = max(0, L - n - window + 1) // 64 if local else 0
            nc = _chunks((L - 1) // 64 - first + 1, aim, most, blocks)
            if nc > 1:
                worst = max(worst, copies * blocks * nc)
    assert got >= 3 * worst * cap * (256 * 4 + 8)  # both kinds write parts of 256 dims


def test_workspace_refuses():
    size = gw.lib().gw_tree_workspace_bytes
    for args in ((0, 2, 64, 16, 32), (8, -1, 64, 16, 32), (8, 2, 0, 16, 32), (8, 2, 1 << 26, 16, 32),
                 (8, 2, 64, 0, 32), (8, 2, 64, 65, 32), (8, 2, 64, 16, 0), (12, 2, 64, 16, 32), (8, 257, 64, 16, 32)):
        assert size(ctypes.byref(_desc()), *args) == 0
        assert gw.last_error().startswith("gw_tree_workspace_bytes:")
    assert size(ctypes.byref(_desc(FOLDED)), 32, 256, 8192, 64, 0) > 1 << 32


# ---- gw_tree_accept, gw_kv_tree_move ----------------------------------------------
def _accept(batch=2, cu=M, lens=M, rows=16, parent=M, draft=M, target=M, path=3 * M, stride=16, n=2 * M, nxt=4 * M,
            new=M, status=0):
    return gw.lib().gw_tree_accept(batch, _at(cu), _at(lens), rows, _at(parent), _at(draft), _at(target), _at(path),
                                   stride, _at(n), _at(nxt) if nxt else None, _at(new) if new else None,
                                   _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=65536), dict(rows=0), dict(rows=65), dict(stride=15), dict(stride=(1 << 40) + 1),
    dict(cu=0), dict(lens=0), dict(parent=0), dict(draft=M + 2), dict(target=0), dict(path=M + 1), dict(n=0), dict(n=M),
    dict(n=3 * M), dict(nxt=3 * M), dict(nxt=2 * M), dict(new=4 * M), dict(new=2 * M), dict(nxt=M + 2), dict(new=M + 1), dict(status=M + 3),
])
def test_accept_refuses(bad):
    assert _accept(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_tree_accept:")


def _move(pools=None, count=None, batch=2, cu=M, lens=M, table=M, pages=64, path=M, stride=16, n=M, status=0):
    pools = pools or [_desc(), _desc(base=2 * M)]
    arr = (gw.PoolDesc * len(pools))(*pools)
    return gw.lib().gw_kv_tree_move(bytes(arr), len(pools) if count is None else count, batch, _at(cu), _at(lens), _at(table),
                                    pages, _at(path), stride, _at(n), _at(status) if status else None, None)


@pytest.mark.parametrize("bad", [
    dict(count=0), dict(count=65), dict(count=-1), dict(pools=[_desc(), _desc(base=0)]), dict(pools=[_desc(), _desc()]),
    dict(pools=[_desc(), _desc(base=2 * M, kvh=8)]), dict(pools=[_desc(), _desc(base=2 * M, dtype=gw.KV_E4M3)]),
    dict(pools=[_desc(FOLDED), _desc(FULL, base=2 * M)]), dict(batch=-1), dict(batch=65536), dict(cu=0),
    dict(lens=M + 1), dict(table=0), dict(pages=0), dict(pages=1 << 27), dict(path=0), dict(stride=0),
    dict(stride=(1 << 40) + 1), dict(n=0), dict(status=M + 2),
])
def test_move_refuses(bad):
    assert _move(**bad) == gw.GW_ERR_INVALID_ARG
    assert gw.last_error().startswith("gw_kv_tree_move:")


def test_commit_empty():
    assert _accept(batch=0, cu=0, path=0) == gw.GW_OK
    assert _move(batch=0, cu=0, path=0) == gw.GW_OK
    assert _move(pools=[_desc(FOLDED, gw.KV_E4M3)]) == gw.GW_ERR_UNSUPPORTED
    assert gw.lib().gw_kv_tree_move(None, 1, 0, None, None, None, 1, None, 1, None, None, None) == gw.GW_ERR_INVALID_ARG


def test_binding_names_missing_tensors():
    for call, name in ((lambda: gw.norm_rope_append(None, None, 1, 1, 1, 1, 1, 1, 1, 1), "q"),
                       (lambda: gw.tree_attn_local(None, 1, 1, 1, 1, 1, 1, None, 1, 32), "pos"),
                       (lambda: gw.tree_attn_local(None, 1, 1, 1, 1, 1, None, 1, 1, 32), "tree_mask"),
                       (lambda: gw.tree_attn_global(None, 1, 1, 1, 1, None, 1, 1), "block_table"),
                       (lambda: gw.tree_accept(1, 1, None, 1, 1, 1, 1), "parent"),
                       (lambda: gw.kv_tree_move([], 1, 1, 1, None, 1), "path")):
        with pytest.raises(gw.GwError, match="%s is None" % name):
            call()
