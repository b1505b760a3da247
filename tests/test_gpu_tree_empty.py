"""Verification calls of a batch all of whose slots are idle: no rows, nothing written, no error."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw

pytestmark = pytest.mark.gpu


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("layout,kv", [("local", 2), ("folded", 1), ("full", 1), ("folded_e4m3", 1)])
def test_no_rows(layout, kv):
    pool = gw.KVPool(layout, "e4m3" if layout == "folded_e4m3" else "bf16", 4, kv)
    dim, rot = (256, 256) if layout == "local" else (512, 128)
    before, status = pool.data.clone(), zeros(1)
    q = torch.empty(0, 8, dim, dtype=torch.bfloat16, device="cuda")
    k, out = torch.empty(0, kv, dim, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)
    w, cs = torch.ones(dim, device="cuda"), torch.zeros(8, rot // 2, 2, device="cuda")
    gw.norm_rope_append(pool, q, k, k, w, w, zeros(0), zeros(0), cs, out, dev_status=status)
    cu, lens, table = zeros(4), torch.tensor([0, 40, 9], dtype=torch.int32, device="cuda"), zeros(3, 3)
    mask, ws = zeros(0, dtype=torch.int64), gw.alloc_workspace_tree(pool, 8, 3, 3, 16, 32)
    if layout == "local":
        gw.tree_attn_local(pool, q, out, cu, lens, table, mask, zeros(0), ws, 32, max_q_rows=16, dev_status=status)
    else:
        gw.tree_attn_global(pool, q, out, cu, lens, table, mask, ws, max_q_rows=16, dev_status=status)
    path, path_lens, nxt, new = zeros(3, 16) - 1, zeros(3) - 1, zeros(3) - 1, zeros(3) - 1
    gw.tree_accept(cu, lens, zeros(0), zeros(0), zeros(0), path, path_lens, nxt, new, dev_status=status)
    gw.kv_tree_move([pool], cu, lens, table, path, path_lens, dev_status=status)
    assert path_lens.tolist() == [0, 0, 0] and new.tolist() == [0, 40, 9]
    assert (path == -1).all() and (nxt == -1).all() and int(status.item()) == 0
    assert torch.equal(pool.data, before)
