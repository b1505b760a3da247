"""One workspace for calls of at most its size: fewer rows, heads, sequences, pages and a smaller window."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,kv,window", [("local", 2, 2000), ("folded", 1, 0), ("full", 1, 0), ("folded_e4m3", 1, 0)])
def test_smaller_calls(layout, kv, window):
    pages = 160
    heads = 16 if layout == "local" else 32
    big = Case(layout, [(2500, 40), (300, 64)], heads, kv, window=window, seed=1)
    ws = gw.alloc_workspace_tree(big.pool, heads, 3, pages, 64, window or 1)  # what a program keeps
    assert big.table.shape[1] <= pages
    want = big.run(max_q_rows=64).clone()
    ws.fill_(0xff)
    assert torch.equal(big.run(max_q_rows=64, ws=ws), want)
    for n, h in ((1, 8), (4, 8), (3, heads), (8, 8), (16, heads)):
        c = Case(layout, [(2500, n), (1300, 1), (64, n)], h, kv, window=window // 2, seed=n)
        want = c.run().clone()
        c.check()
        ws.fill_(0xff)  # no call needs what another left
        assert torch.equal(c.run(ws=ws), want)
