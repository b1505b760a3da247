"""Logits that are infinite: a visible one of minus infinity has weight 0, one of plus
infinity or NaN makes its row and head NaN; on e4m3 pools any infinity in q does."""

import numpy as np
import pytest
import torch

from tests.tree_helpers import Case, kv_rows, to64

pytestmark = pytest.mark.gpu

BF16 = [("local", "bf16"), ("folded", "bf16"), ("full", "bf16")]
E4M3 = [("local", "e4m3"), ("folded_e4m3", "")]
INF = float("inf")


def put_k(c, b, token, dim, value):
    """Element `dim` (below 128: rotated, not V's) of K of a token, all heads."""
    page, off = int(c.table[b, token // 16]), token % 16
    if c.layout == "local":
        c.cells[page, :, 0, off, dim] = value
    else:
        cb = dim // 8 + (64 if c.layout == "folded" else 0)
        c.cells[page, off // 8, cb, off % 8, dim % 8] = value


def compare(c):
    """Every row and head by the definition, with the infinities of float64."""
    got = to64(c.out)
    for b, (L, n) in enumerate(c.plan):
        base, pos = L - n, c.pos[c.cu[b]:c.cu[b + 1]].astype(np.int64)
        lo = max(0, base - c.window + 1) if c.window else 0
        sees = np.concatenate([np.ones((n, base - lo), bool), c.sees[b]], 1)
        if c.window:
            sees &= np.concatenate([np.arange(lo, base), pos])[None] > pos[:, None] - c.window
        k, v = kv_rows(c.cells, c.layout, c.table[b], np.arange(lo, L))
        q = to64(c.q[c.cu[b]:c.cu[b + 1]])
        for r in range(n):
            for h in range(c.heads):
                kv = h // (c.heads // k.shape[0])
                with np.errstate(invalid="ignore"):
                    e = (k[kv][sees[r]] * q[r, h]).sum(-1) * c.scale
                g = got[c.cu[b] + r, h]
                if np.isnan(e).any() or (e == INF).any():
                    assert np.isnan(g).all(), (b, r, h)
                    continue
                keep = e > -INF
                if not keep.any():
                    assert (g == 0).all(), (b, r, h)
                    continue
                p = np.exp(e[keep] - e[keep].max())
                p /= p.sum()
                vv = v[kv][sees[r]][keep]
                want, size = p @ vv, p @ np.abs(vv)
                assert (np.abs(g - want) <= 2.0 ** -8 * (2 * size + np.abs(want)) * 1.05 + 1e-6).all(), (b, r, h)


@pytest.mark.parametrize("layout,dtype", BF16)
@pytest.mark.parametrize("n", [3, 8, 20])  # few rows and many
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("L", [300, 1500])  # one chunk of a global cache and several
def test_k(layout, dtype, n, value, L):
    """The heads of one sign of q get NaN, those of the other leave the token out."""
    local = layout == "local"
    c = Case(layout, [(L, n), (70, 2)], 8, 2 if local else 1, dtype, window=250 if local else 0, seed=n)
    put_k(c, 0, L - n - 30, 5, value)  # seen by every row
    put_k(c, 0, L - 1, 70, -value)     # the last draft
    c.run()
    assert int(c.status.item()) == 0
    compare(c)
    seen = torch.isnan(c.out[:n]).any(-1)
    assert seen.any() and not seen.all()


@pytest.mark.parametrize("layout,dtype", BF16)
@pytest.mark.parametrize("rows", [1, 64])  # the call's bound: few rows and many
def test_only_minus_infinity(layout, dtype, rows):
    """Rows all of whose logits are minus infinity are zeros, as rows that see nothing."""
    local = layout == "local"
    c = Case(layout, [(1, 1), (1, 1), (600, 1)], 8, 2 if local else 1, dtype, window=600 if local else 0, seed=3)
    for b, (L, _) in enumerate(c.plan):
        for t in range(L):
            put_k(c, b, t, 9, 1.0 if b != 1 else -1.0)
    c.q[:, :, 9] = -INF
    c.run(max_q_rows=rows)
    assert (c.out[0] == 0).all() and torch.isnan(c.out[1]).all() and (c.out[2] == 0).all()
    compare(c)


@pytest.mark.parametrize("layout,dtype", E4M3)
@pytest.mark.parametrize("rows", [1, 64])
@pytest.mark.parametrize("value", [INF, -INF])
def test_q_on_e4m3(layout, dtype, rows, value):
    local = layout == "local"
    c = Case(layout, [(1, 1), (600, 1), (2, 1)], 8, 2 if local else 1, dtype or "bf16", window=600 if local else 0, seed=3)
    good = c.run(max_q_rows=rows).clone()
    c.q[0, 1, 9] = c.q[1, 6, 200] = value
    out = c.run(max_q_rows=rows)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[1, 6]).all()
    out[0, 1], out[1, 6] = good[0, 1], good[1, 6]
    assert torch.equal(out, good)
