"""Drafted trees over infinities and NaN: they reach the rows that see them and no others."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import Case

pytestmark = pytest.mark.gpu

POOLS = [("local", "bf16"), ("local", "e4m3"), ("folded", "bf16"), ("full", "bf16"), ("folded_e4m3", "")]


def case(layout, dtype, n, seed, L=600):
    local = layout == "local"
    return Case(layout, [(70, 3), (L, n)], 8, 2 if local else 1, dtype or "bf16", window=L // 2 if local else 0, seed=seed)


@pytest.mark.parametrize("layout,dtype", POOLS)
@pytest.mark.parametrize("n,L", [(4, 600), (8, 600), (24, 600), (40, 600), (4, 5000), (24, 5000)])  # few rows and many
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_q(layout, dtype, n, L, value):
    c = case(layout, dtype, n, 3, L)
    good = c.run().clone()
    c.q[5, 2, 130] = value
    out = c.run()
    assert torch.isnan(out[5, 2]).all() and int(c.status.item()) == 0
    good[5, 2] = out[5, 2] = 0
    assert torch.equal(out, good)


@pytest.mark.parametrize("layout,dtype", POOLS)
@pytest.mark.parametrize("n,L", [(4, 600), (8, 600), (24, 600), (40, 600), (4, 5000), (24, 5000)])
def test_k_of_a_draft(layout, dtype, n, L):
    """A leaf's K is NaN: the other rows do not see it."""
    c = case(layout, dtype, n, 4, L)
    c.sees[1][:, n - 1] = False
    c.sees[1][n - 1, n - 1] = True
    c.mask[3:] &= (1 << (n - 1)) - 1
    c.mask[3 + n - 1] |= 1 << (n - 1)
    good = c.run().clone()
    c.check()
    page, off = int(c.table[1, (L - 1) // 16]), (L - 1) % 16
    raw = c.cells.view(torch.uint8 if c.cells.dtype != torch.bfloat16 else torch.int16)
    nan = 0x7f if raw.dtype == torch.uint8 else 0x7fc0
    if layout == "local":
        raw[page, :, 0, off] = nan
    else:  # a rotated dim, which is not V's
        raw[page, off // 8, {"folded": 64, "full": 0, "folded_e4m3": 32}[layout], off % 8] = nan
    out = c.run()
    assert torch.equal(out[:-1], good[:-1]) and torch.isnan(out[-1]).all()


@pytest.mark.parametrize("layout,dtype", POOLS)
@pytest.mark.parametrize("n", [4, 24])
def test_rows_behind_the_last_sequence(layout, dtype, n):
    c = case(layout, dtype, n, 6)
    good = c.run().clone()
    full = torch.full((c.rows + 5, 8, c.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    q, d = torch.cat([c.q, c.q[:5]]), c.dev
    mask = torch.cat([d["mask"], d["mask"][:5]])
    if layout == "local":
        gw.tree_attn_local(c.pool, q, full, d["cu"], d["lens"], d["table"], mask, torch.cat([d["pos"], d["pos"][:5]]),
                           c.ws, c.window, max_q_rows=n)
    else:
        gw.tree_attn_global(c.pool, q, full, d["cu"], d["lens"], d["table"], mask, c.ws, max_q_rows=n)
    assert torch.equal(full[:c.rows], good) and (full[c.rows:] == 7).all()
