"""Drafted trees whose block tables name pages that do not exist: such a page counts
as zeros, by value, wherever it lies and whatever its buffer held before."""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import PAGE, Case, attend, kv_rows, to64

pytestmark = pytest.mark.gpu

POOLS = [("local", "bf16"), ("local", "e4m3"), ("folded", "bf16"), ("full", "bf16"), ("folded_e4m3", "")]


class BadPages(Case):
    """Case whose table entries bad[(sequence, logical page)] are replaced on the device."""

    def table_with(self, bad):
        table = self.table.copy()
        for (b, p), entry in bad.items():
            table[b, p] = entry
        return torch.from_numpy(table).cuda()

    def compare(self, bad):
        got = to64(self.out)
        for b, (L, n) in enumerate(self.plan):
            base, pos = L - n, self.pos[self.cu[b]:self.cu[b + 1]].astype(np.int64)
            lo = max(0, base - self.window + 1) if self.window else 0
            t = np.arange(lo, L)
            sees = np.concatenate([np.ones((n, base - lo), bool), self.sees[b]], 1)
            if self.window:
                sees &= np.concatenate([np.arange(lo, base), pos])[None] > pos[:, None] - self.window
            k, v = kv_rows(self.cells, self.layout, self.table[b], t)
            gone = np.isin(t // PAGE, [p for s, p in bad if s == b])
            k[:, gone], v[:, gone] = 0, 0
            want, size = attend(to64(self.q[self.cu[b]:self.cu[b + 1]]), k, v, sees, self.scale)
            # the weights' rounding in numerator and denominator, and the output's: 2^-8 each
            tol = 2.0 ** -8 * (2 * size + np.abs(want)) * 1.05 + 1e-6
            g = got[self.cu[b]:self.cu[b + 1]]
            assert np.isfinite(g).all() and (np.abs(g - want) <= tol).all(), (b, float((np.abs(g - want) / tol).max()))


@pytest.mark.parametrize("layout,dtype", POOLS)
@pytest.mark.parametrize("n", [2, 4, 8, 12, 40])  # few rows and many
@pytest.mark.parametrize("where", ["middle", "tile", "drafts", "many"])
def test_counts_as_zeros(layout, dtype, n, where):
    local = layout == "local"
    # pages of 16, tiles of up to 128 tokens, up to three buffers: page 45 is in a buffer that has been used
    c = BadPages(layout, [(1100, n), (130 + n, n)], 8, 2 if local else 1, dtype or "bf16",
                 window=1000 if local else 0, seed=n, sigma=1.0)
    last = 1099 // PAGE
    bad = {"middle": {(0, 45): -1, (1, 3): c.pages},
           "tile": {(0, p): c.pages + p for p in range(40, 56)},
           "drafts": {(0, last): -5, (1, (129 + n) // PAGE): 1 << 30},
           "many": {(0, p): -1 for p in range(9, last, 3)}}[where]
    # K twice as large there as elsewhere would show: the rows that are left out are not small
    c.run(table=c.table_with(bad))
    assert int(c.status.item()) == gw.GW_DEV_PAGE_RANGE
    c.compare(bad)


@pytest.mark.parametrize("layout,dtype", POOLS)
@pytest.mark.parametrize("n", [4, 12])
def test_no_page_at_all(layout, dtype, n):
    """Every page refused: all logits 0, all values 0."""
    local = layout == "local"
    c = BadPages(layout, [(300, n), (300, n)], 8, 2 if local else 1, dtype or "bf16", window=200 if local else 0, seed=1)
    bad = {(1, p): -1 for p in range(19)}
    c.run(table=c.table_with(bad))
    assert int(c.status.item()) == gw.GW_DEV_PAGE_RANGE
    c.compare(bad)
    assert (c.out[n:] == 0).all()
