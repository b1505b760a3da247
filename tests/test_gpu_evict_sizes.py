"""gw_kv_evict_select and gw_kv_evict_compact at the longest sequences that they
accept, where indices reach 2^31, and where their pipelines run for many steps."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

GUARD = 1 << 16  # elements before a row


def _guarded(n, dtype, fill):
    flat = torch.empty(GUARD + n + GUARD, dtype=dtype, device="cuda")
    flat[:GUARD].fill_(fill)
    flat[GUARD + n:].fill_(fill)
    return flat, flat[GUARD:GUARD + n].view(1, n)


def _guards_hold(flat, fill):
    return bool((flat[:GUARD] == fill).all()) and bool((flat[-GUARD:] == fill).all())


def _pieces(n, step=1 << 28):
    return [slice(i, min(n, i + step)) for i in range(0, n, step)]


def test_select_keeps_all_of_the_longest_row():
    """2^31 - 1 tokens within the budget."""
    n = 2 ** 31 - 1
    flat, keep = _guarded(n, torch.int32, -9)
    acc, lens = torch.empty(1, n, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_evict_select(acc, G.i32([n]), n, keep, lens)
    assert int(lens) == n and _guards_hold(flat, -9)
    for p in _pieces(n):
        assert torch.equal(keep[0, p], torch.arange(p.start, p.stop, dtype=torch.int32, device="cuda"))


def test_compact_weights_of_the_longest_sequence():
    """The most pages that a sequence has; the weights behind the kept ones
    become 0.  All rows stay in place (every table entry is the one page)."""
    pages = 2 ** 27 - 1
    n = 16 * pages
    kept = n - 5
    pool = gw.KVPool("folded_e4m3", "e4m3", 1)
    before = pool.data.clone()
    flat, acc = _guarded(n, torch.float32, 7.0)
    acc.fill_(1.0)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    keep = torch.arange(kept, dtype=torch.int32, device="cuda").view(1, kept)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_evict_compact(pool, table, G.i32([n]), keep, G.i32([kept]), acc, dev_status=status)
    assert int(status) == 0 and _guards_hold(flat, 7.0) and torch.equal(pool.data, before)
    for p in _pieces(kept):
        assert bool((acc[0, p] == 1).all())
    assert bool((acc[0, kept:] == 0).all())
