"""The merge of a tree's chunks is the same however many sequences the call has."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import Case, to64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,dtype,heads,kv,n", [("folded", "bf16", 8, 1, 4), ("full", "bf16", 8, 1, 8),
                                                     ("folded_e4m3", "", 16, 1, 2), ("folded", "bf16", 32, 1, 5),
                                                     ("local", "bf16", 8, 4, 3), ("local", "e4m3", 8, 2, 20)])
def test_large_batches(layout, dtype, heads, kv, n):
    long = 2700 if layout == "local" or n == 5 else 1500  # several chunks each
    plan = [(long + 13 * b, n) for b in range(70)]
    window = 5000 if layout == "local" else 0
    c = Case(layout, plan, heads, kv, dtype or "bf16", window=window, seed=n)
    whole = c.run().clone()
    assert int(c.status.item()) == 0
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    for b in (0, 33, 69):
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        q, out = c.q[rows].contiguous(), torch.empty_like(c.q[rows])
        table, mask = i32(c.table[b:b + 1].tolist()), torch.from_numpy(c.mask[rows]).cuda()
        ws = gw.alloc_workspace_tree(c.pool, heads, 1, table.shape[1], n, window or 1)
        if layout == "local":
            gw.tree_attn_local(c.pool, q, out, i32([0, n]), i32([plan[b][0]]), table, mask, i32(c.pos[rows].tolist()),
                               ws, window, max_q_rows=n)
        else:
            gw.tree_attn_global(c.pool, q, out, i32([0, n]), i32([plan[b][0]]), table, mask, ws, max_q_rows=n)
        assert torch.equal(out, whole[rows]), b
        want, size = c.want(b)
        tol = 2.0 ** -8 * (2 * size + abs(want)) * 1.05 + 1e-6  # as Case.check
        assert (abs(to64(out) - want) <= tol).all(), b
