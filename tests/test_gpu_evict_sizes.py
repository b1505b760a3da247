"""gw_kv_evict_select and gw_kv_evict_compact at the longest sequences that they
accept, where indices reach 2^31, and where their pipelines run for many steps."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G
from tests.test_gpu_acc import Cache

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


ROW = {"folded": 80, "full": 128, "folded_e4m3": 40}  # 16-byte column blocks of a row


def _cut(L, share, g):
    """A random choice of L * share tokens (L - 1 for "all but one"), ascending."""
    n = L - 1 if share == "all but one" else int(L * share)
    return torch.randperm(L, generator=g, device="cuda")[:n].sort().values.to(torch.int32)


@pytest.mark.parametrize("layout", ["folded", "full", "folded_e4m3"])
@pytest.mark.parametrize("batch", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("share", [0.25, 15 / 16, "all but one"])
@pytest.mark.parametrize("other_pages", [False, True])
def test_long_cuts(layout, batch, share, other_pages):
    """Walks of many steps, over blocks and over clusters of every size that
    the batches get, with a partial last step: every byte of the pool, every
    weight."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    lens = [70001 - 7777 * b for b in range(batch)]
    width = (max(lens) + 15) // 16 + 1
    need = [(n + 15) // 16 for n in lens]
    copies = 2 if other_pages else 1
    perm = torch.randperm(copies * sum(need), generator=g, device="cuda").to(torch.int32)
    pool = gw.KVPool(layout, "e4m3" if layout == "folded_e4m3" else "bf16", copies * sum(need))
    pool.data.copy_(torch.randint(0, 256, (pool.nbytes,), generator=g, device="cuda", dtype=torch.uint8))
    tables = torch.full((copies, batch, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for c in range(copies):
        for b in range(batch):
            tables[c, b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
    keeps = [_cut(n, share, g) for n in lens]
    keep = torch.full((batch, max(len(k) for k in keeps) + 3), -5, dtype=torch.int32, device="cuda")
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    acc = torch.rand(batch, width * 16 + 1, generator=g, device="cuda")
    want, before, old = pool.data.clone(), pool.data.clone(), acc.clone()
    rows = [t.view(-1, 2, ROW[layout], 8, 16) for t in (want, before)]
    for b, k in enumerate(keeps):
        j, i = k.long(), torch.arange(len(k), device="cuda")
        src, dst = tables[0, b].long()[j // 16], tables[-1, b].long()[i // 16]
        rows[0][dst, i % 16 // 8, :, i % 8] = rows[1][src, j % 16 // 8, :, j % 8]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_evict_compact(pool, tables[0], G.i32(lens), keep, G.i32([len(k) for k in keeps]), acc,
                        tables[1] if other_pages else None, status)
    assert int(status) == 0 and torch.equal(pool.data, want)
    for b, k in enumerate(keeps):
        assert torch.equal(acc[b, :len(k)], old[b, k.long()])
        assert bool((acc[b, len(k):lens[b]] == 0).all()) and torch.equal(acc[b, lens[b]:], old[b, lens[b]:])


@pytest.mark.parametrize("layout", ["folded", "full", "folded_e4m3"])
@pytest.mark.parametrize("lens,heads,ctas", [([20001, 300, 8192], 8, 2), ([8192 - 37 * b for b in range(16)], 32, 0),
                                             ([6000], 16, 1)])
def test_weights_of_many_tiles_a_block(layout, lens, heads, ctas):
    """Blocks of the weights pass that go through more tiles than they have
    stages; the bits do not depend on the CTA cap."""
    c = Cache(layout, lens, heads)
    acc = c.new_acc(0.25)
    old = acc.clone()
    try:
        gw.set_max_ctas(ctas)
        out, lse = c.run(acc)
    finally:
        gw.set_max_ctas(0)
    assert int(c.status) == 0
    c.check(out, lse, acc, old)
    again = old.clone()
    out2, lse2 = c.run(again)
    assert torch.equal(again, acc) and torch.equal(out2, out) and torch.equal(lse2, lse)


def test_entries_below_their_place_stay():
    """Behind an entry that is skipped others can ascend and still lie below
    their own place: they are skipped too, with their weights."""
    c = Cache("folded", [100] * 4, 8)
    keeps = [[5, 0, 1, 9], [-1, 0, 2, 3], [0, 1, 0, 1], [-3, -2, -1, 50]]
    moves = [{0: 5, 3: 9}, {2: 2, 3: 3}, {0: 0, 1: 1}, {3: 50}]
    before = c.pool.data.clone()
    acc = torch.rand(4, c.width * 16, device="cuda")
    want, old = acc.clone(), acc.clone()
    gw.kv_evict_compact(c.pool, c.bt, c.n, torch.tensor(keeps, dtype=torch.int32, device="cuda"), G.i32([4] * 4), acc,
                        dev_status=c.status)
    assert int(c.status) == gw.GW_DEV_KEEP_RANGE
    expect, src = before.clone().view(-1, 2, 80, 8, 16), before.view(-1, 2, 80, 8, 16)
    for b, m in enumerate(moves):
        for i, j in m.items():
            expect[int(c.table[b, i // 16]), i % 16 // 8, :, i % 8] = src[int(c.table[b, j // 16]), j % 16 // 8, :, j % 8]
            want[b, i] = old[b, j]
        want[b, 4:100] = 0
    assert torch.equal(c.pool.data, expect.reshape(-1)) and torch.equal(acc, want)


@pytest.mark.parametrize("layout,batch", [("folded", 1), ("folded", 4), ("full", 2), ("folded_e4m3", 3)])
@pytest.mark.parametrize("share", [0.25, "all but one"])
def test_moves_under_a_cta_cap(layout, batch, share):
    """Few blocks that take the walks in turn, and clusters that do: the same
    bytes and weights."""
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [9001 - 1111 * b for b in range(batch)]
    need = [(n + 15) // 16 for n in lens]
    pool = gw.KVPool(layout, "e4m3" if layout == "folded_e4m3" else "bf16", sum(need))
    start = torch.randint(0, 256, (pool.nbytes,), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.full((batch, max(need)), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    keep = torch.full((batch, max(lens)), -5, dtype=torch.int32, device="cuda")
    n = []
    for b in range(batch):
        table[b, :need[b]] = perm[sum(need[:b]):sum(need[:b + 1])]
        k = _cut(lens[b], share, g)
        keep[b, :len(k)] = k
        n.append(len(k))
    weights = torch.rand(batch, 16 * max(need), generator=g, device="cuda")
    got = []
    try:
        for cap in (0, 1, 7, 50, 100, 130):
            pool.data.copy_(start)
            acc = weights.clone()
            gw.set_max_ctas(cap)
            gw.kv_evict_compact(pool, table, G.i32(lens), keep, G.i32(n), acc)
            got.append((pool.data.clone(), acc))
    finally:
        gw.set_max_ctas(0)
    for data, acc in got[1:]:
        assert torch.equal(data, got[0][0]) and torch.equal(acc, got[0][1])


def test_the_cta_cap_holds_for_moves():
    """One block takes all 164 walks of four sequences in turn: many times the
    time that they take at once."""
    g = torch.Generator(device="cuda").manual_seed(3)
    L, batch = 8192, 4
    pool = gw.KVPool("folded", "bf16", batch * L // 16)
    table = torch.arange(batch * L // 16, dtype=torch.int32, device="cuda").view(batch, -1)
    keep = torch.stack([_cut(L, 0.5, g) for _ in range(batch)])
    acc, lens, n = torch.rand(batch, L, device="cuda"), G.i32([L] * batch), G.i32([L // 2] * batch)
    times = []
    try:
        for cap in (0, 1):
            gw.set_max_ctas(cap)
            for _ in range(2):
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                torch.cuda.synchronize()
                a.record()
                gw.kv_evict_compact(pool, table, lens, keep, n, acc)
                b.record()
                torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
    finally:
        gw.set_max_ctas(0)
    assert times[1] > 8 * times[0], times
