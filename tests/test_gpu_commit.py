"""gw_tree_accept and gw_kv_tree_move against a walk and moves in Python."""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import PAGE, new_pool, tree_of

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def walk(parent, draft, target):
    path = [0]
    while True:
        at = path[-1]
        nxt = [i for i in range(1, len(parent)) if parent[i] == at and 0 <= parent[i] < i and draft[i] == target[at]]
        if not nxt:
            return path
        path.append(nxt[0])


def step(rng, sizes, vocab):
    """Trees of these sizes; the smaller the vocabulary, the more drafts meet the target's choice."""
    trees = [tree_of(rng, n) if n else [] for n in sizes]
    rows = sum(sizes)
    return trees, rng.integers(0, vocab, rows), rng.integers(0, vocab, rows), np.concatenate([[0], np.cumsum(sizes)])


@pytest.mark.parametrize("vocab", [1, 2, 5, 1000])
@pytest.mark.parametrize("sizes", [[1], [2, 64, 1, 0, 33], [64] * 9, [5] * 130])
def test_accept(sizes, vocab):
    rng = np.random.default_rng(vocab + len(sizes))
    trees, draft, target, cu = step(rng, sizes, vocab)
    lens = np.array([n + int(rng.integers(0, 2 ** 31 - 100)) for n in sizes])
    batch, most = len(sizes), max(sizes)
    path = torch.full((batch, 70), -5, dtype=torch.int32, device="cuda")
    n, nxt, new = (torch.full((batch,), -9, dtype=torch.int32, device="cuda") for _ in range(3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.tree_accept(i32(cu), i32(lens), i32([p for t in trees for p in t]), i32(draft), i32(target), path, n, nxt, new,
                   max_q_rows=most, dev_status=status)
    assert int(status.item()) == 0
    path, n, nxt, new = path.cpu().numpy(), n.cpu().numpy(), nxt.cpu().numpy(), new.cpu().numpy()
    for b, size in enumerate(sizes):
        if size == 0:
            assert n[b] == 0 and nxt[b] == -9 and new[b] == lens[b] and (path[b] == -5).all()
            continue
        d, t = draft[cu[b]:cu[b + 1]], target[cu[b]:cu[b + 1]]
        want = walk(trees[b], d, t)
        assert list(path[b, :n[b]]) == want and (path[b, n[b]:] == -5).all()
        assert nxt[b] == t[want[-1]] and new[b] == lens[b] - size + len(want)


def test_accept_bad_trees():
    """Parents that are not before their row are never followed; sizes that do not fit are refused."""
    parent = [-1, 0, 5, 1, -3, 4, 2 ** 31 - 1] + [77, 0] + [-1, 0, 0]
    draft, target = [1] * 12, [1] * 12
    cu, lens = [0, 7, 9, 12], [20, 1, 12]
    path = torch.full((3, 8), -5, dtype=torch.int32, device="cuda")
    n = torch.full((3,), -9, dtype=torch.int32, device="cuda")
    seq, status = i32(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.tree_accept(i32(cu), seq, i32(parent), i32(draft), i32(target), path, n, new_lens=seq, dev_status=status)
    assert int(status.item()) == gw.GW_DEV_TREE_RANGE | gw.GW_DEV_LEN_RANGE
    # sequence 0: row 5's parent 4 is reachable only from itself; the root's own parent is not read
    assert n.tolist() == [3, 0, 2] and path[0, :3].tolist() == [0, 1, 3] and path[2, :2].tolist() == [0, 1]
    assert seq.tolist() == [16, 1, 11]
    status.zero_()
    gw.tree_accept(i32(cu), i32(lens), i32(parent), i32(draft), i32(target), path, n, max_q_rows=3, dev_status=status)
    assert int(status.item()) == gw.GW_DEV_LEN_RANGE and n.tolist() == [0, 0, 2]


def moved(pools, cu, lens, table, path, n):
    """The pools' bytes [pages, 16 tokens, ...] after the moves, by token."""
    for x in pools:
        for b in range(len(lens)):
            base = lens[b] - (cu[b + 1] - cu[b])
            for i in range(n[b]):
                s, d = base + path[b][i], base + i
                x[table[b][d // PAGE], d % PAGE] = x[table[b][s // PAGE], s % PAGE].copy()
    return pools


def by_token(pool, layout, kv):
    """A pool's bytes as [pages, 16, bytes of a token]."""
    x = pool.data.cpu().numpy()
    if layout == "local":
        return x.reshape(pool.num_pages, kv * 2, PAGE, -1).transpose(0, 2, 1, 3).reshape(pool.num_pages, PAGE, -1)
    return x.reshape(pool.num_pages, 2, -1, 8, 16).transpose(0, 1, 3, 2, 4).reshape(pool.num_pages, PAGE, -1)


def plan(rng, sizes):
    lens = [n + int(rng.integers(0, 60)) for n in sizes]
    need = [-(-L // PAGE) for L in lens]
    perm = rng.permutation(sum(need) + 2)
    table, at = np.full((len(sizes), max(need + [1]) + 1), -1), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return lens, table, len(perm)


@pytest.mark.parametrize("layout,kv,dtype", [("local", 1, "bf16"), ("local", 16, "bf16"), ("local", 3, "e4m3"),
                                             ("folded", 1, "bf16"), ("full", 1, "bf16"), ("folded_e4m3", 1, "e4m3")])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 64, 17, 2], [64, 64, 31]])
def test_move(layout, kv, dtype, sizes):
    rng = np.random.default_rng(len(sizes) + kv)
    lens, table, pages = plan(rng, sizes)
    cu = np.concatenate([[0], np.cumsum(sizes)])
    path, n = np.full((len(sizes), 64), -1), []
    for b, size in enumerate(sizes):
        m = int(rng.integers(1, size + 1)) if size else 0
        n.append(m)
        if m:
            path[b, :m] = np.concatenate([[0], np.sort(rng.choice(np.arange(1, size), m - 1, replace=False))])
    pools = []
    for i in range(3):
        pool, _ = new_pool(layout, pages + i, kv, dtype)
        pool.data.copy_(torch.from_numpy(rng.integers(0, 256, pool.data.numel(), dtype=np.uint8)))
        pools.append(pool)
    want = moved([by_token(p, layout, kv) for p in pools], cu, lens, table, path, n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_tree_move(pools, i32(cu), i32(lens), i32(table), i32(path), i32(n), dev_status=status)
    assert int(status.item()) == 0
    for p, w in zip(pools, want):
        assert np.array_equal(by_token(p, layout, kv), w)


def test_move_skips_what_does_not_fit():
    sizes = [6, 6, 6, 6, 6]
    rng = np.random.default_rng(1)
    lens, table, pages = plan(rng, sizes)
    cu = np.arange(6) * 6
    path = np.tile(np.array([0, 2, 3, 5, -1, -1]), (5, 1))
    n = [4, 7, 4, 4, 4]                    # sequence 1: longer than its rows
    path[2, :4] = [0, 4, 4, 5]             # one not above the one before it
    path[3, :4] = [0, 1, 6, 3]             # one outside, one that stays
    table[4, :] = pages + 3                # pages outside
    pool, _ = new_pool("folded", pages)
    pool.data.copy_(torch.from_numpy(rng.integers(0, 256, pool.data.numel(), dtype=np.uint8)))
    want = by_token(pool, "folded", 1)
    moved([want], cu, lens, table, [[0, 2, 3, 5], [], [0, 4], [0, 1], []], [4, 0, 2, 2, 0])
    base = lens[2] - 6
    want[table[2][(base + 3) // PAGE], (base + 3) % PAGE] = want[table[2][(base + 5) // PAGE], (base + 5) % PAGE]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_tree_move([pool], i32(cu), i32(lens), i32(table), i32(path), i32(n), dev_status=status)
    assert int(status.item()) == gw.GW_DEV_TREE_RANGE | gw.GW_DEV_PAGE_RANGE
    assert np.array_equal(by_token(pool, "folded", 1), want)
    for bad in ([5] + lens[1:], [table.shape[1] * 16 + 1] + lens[1:]):
        status.zero_()
        gw.kv_tree_move([pool], i32(cu[:2]), i32(bad[:1]), i32(table[:1]), i32(path[:1]), i32(n[:1]), dev_status=status)
        assert int(status.item()) == gw.GW_DEV_LEN_RANGE
    assert np.array_equal(by_token(pool, "folded", 1), want)


def test_many_pools_of_which_one_is_large():
    """64 pools in a call; one of more than 2^32 bytes, rows in its last pages."""
    pages = (1 << 32) // 20480 + 6
    big = gw.KVPool("folded", "bf16", pages)
    small = [gw.KVPool("folded", "bf16", 8) for _ in range(2)]
    cells = big.data.view(torch.uint8).view(pages, 2, 80, 8, 16)
    cells[pages - 2:].copy_(torch.randint(0, 256, (2, 2, 80, 8, 16), dtype=torch.uint8, device="cuda"))
    table = i32([[pages - 1, pages - 2]])
    row = cells[pages - 2, 0, :, 3].clone()   # token 19
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_tree_move([big], i32([0, 8]), i32([20]), table, i32([[0, 7]]), i32([2]), dev_status=status)
    assert int(status.item()) == 0 and torch.equal(cells[pages - 1, 1, :, 5], row)   # token 13
    pools = [gw.KVPool("folded", "bf16", 2) for _ in range(64)]
    for i, p in enumerate(pools):
        p.data.fill_(i)
        p.data.view(2, 2, 80, 8, 16)[1, 0, :, 3] = 200
    gw.kv_tree_move(pools, i32([0, 8]), i32([20]), i32([[0, 1]]), i32([[0, 7]]), i32([2]), dev_status=status)
    for i, p in enumerate(pools):
        x = p.data.view(2, 2, 80, 8, 16)
        assert (x[0, 1, :, 5] == 200).all() and int((x == 200).sum()) == 2 * 80 * 16 and int((x == i).sum()) > 0
    # the table names pages that the small pools do not have
    gw.kv_tree_move(small, i32([0, 8]), i32([20]), table, i32([[0, 7]]), i32([2]), dev_status=status)
    assert int(status.item()) == gw.GW_DEV_PAGE_RANGE


def test_binding_refuses():
    v = i32([0, 0])
    path = i32([[0, 1]])
    with pytest.raises(gw.GwError):
        gw.tree_accept(i32([0, 2]), i32([2]), v, v[:1], v, path, i32([0]))
    with pytest.raises(gw.GwError):
        gw.tree_accept(i32([0, 2]), i32([2]), v, v, v, path, i32([0]), max_q_rows=3)
    with pytest.raises(gw.GwError):
        gw.tree_accept(i32([0, 2]), i32([2]), v, v, v, path.t(), i32([0]))
    with pytest.raises(gw.GwError):
        gw.kv_tree_move([], i32([0, 2]), i32([2]), path, path, i32([1]))
    pools = [gw.KVPool("folded", "bf16", 2), gw.KVPool("full", "bf16", 2)]
    with pytest.raises(gw.GwError, match="differs"):
        gw.kv_tree_move(pools, i32([0, 2]), i32([2]), path, path, i32([1]))
