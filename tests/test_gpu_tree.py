"""gw_tree_attn_local and gw_tree_attn_global against attention by its
definition in float64: head layouts, lengths, windows, masks, pool types."""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import Case

pytestmark = pytest.mark.gpu

# lengths around pages, tiles of 64 and chunks of 256, with rows up to the length
EDGES = [(1, 1), (5, 5), (16, 3), (17, 17), (0, 0), (64, 64), (65, 1), (63, 5), (81, 64), (257, 2), (300, 33), (128, 16)]


def at_most(plan, rows):
    return [(L, min(n, rows)) for L, n in plan]


# rows x heads of a KV head: up to 16, up to 32, more
@pytest.mark.parametrize("most", [16, 32, 512])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv", [(4, 4), (8, 4), (8, 2), (16, 2), (1, 1), (8, 1)])
def test_local_edges(heads, kv, dtype, most):
    c = Case("local", at_most(EDGES, most * kv // heads), heads, kv, dtype, window=64, seed=heads * 10 + kv)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 5, 17, 64, 100, 1024, 2 ** 31 - 1])
@pytest.mark.parametrize("rows", [8, 16, 64])
def test_local_windows(window, dtype, rows):
    plan = at_most([(40, 9), (700, 20), (1300, 64), (64, 64), (130, 2)], rows)
    c = Case("local", plan, 4, 2, dtype, window=window, seed=window % 97)
    c.run()
    c.check()


@pytest.mark.parametrize("layout", ["folded", "full", "folded_e4m3"])
@pytest.mark.parametrize("heads", [8, 16, 32])
@pytest.mark.parametrize("most", [32, 64, 2048])
def test_global_edges(layout, heads, most):
    c = Case(layout, at_most(EDGES, most // heads), heads, seed=heads)
    c.run()
    c.check()


@pytest.mark.parametrize("layout,rows", [("local", 4), ("local", 8), ("local", 64), ("folded", 64), ("full", 64),
                                         ("folded_e4m3", 64), ("folded", 4), ("full", 4), ("folded_e4m3", 4),
                                         ("folded", 8), ("full", 8), ("folded_e4m3", 8)])
def test_any_words(layout, rows):
    """Words that are no trees, rows that see no draft, and sequences without a cache before them."""
    c = Case(layout, at_most([(7, 7), (64, 64), (200, 30), (33, 1), (1, 1), (1100, 5)], rows), 8,
             2 if layout == "local" else 1, window=90 if layout == "local" else 0, sees="any", seed=5)
    c.sees[4][:] = False
    c.mask[c.cu[4]] = 0
    c.run()
    c.check()
    assert (c.out[c.cu[4]:c.cu[5]] == 0).all()


@pytest.mark.parametrize("layout,heads,n", [("folded", 32, 5), ("folded", 8, 17), ("full", 16, 9), ("folded_e4m3", 32, 4),
                                            ("folded_e4m3", 8, 64), ("folded", 8, 4), ("folded", 32, 1),
                                            ("full", 16, 2), ("folded_e4m3", 8, 3), ("folded_e4m3", 32, 1),
                                            ("folded", 32, 2), ("folded", 8, 7), ("full", 16, 4), ("full", 32, 2),
                                            ("folded", 16, 3), ("folded_e4m3", 32, 2)])
def test_global_chunks(layout, heads, n):
    """Several chunks, an odd last one among them."""
    c = Case(layout, [(511, n), (513, n), (2600, n), (1024 + n, n)], heads, seed=n)
    c.run()
    c.check()


@pytest.mark.parametrize("layout,dtype,rows", [("local", "bf16", 40), ("local", "bf16", 4), ("local", "e4m3", 40),
                                               ("local", "e4m3", 4), ("folded", "bf16", 40), ("folded", "bf16", 3),
                                               ("full", "bf16", 4), ("folded_e4m3", "", 40), ("folded_e4m3", "", 4),
                                               ("folded", "bf16", 8), ("full", "bf16", 7)])
def test_long_chunks(layout, dtype, rows):
    """Sequences with as many chunks as there may be, and longer ones; rows in many blocks."""
    L = 46000 if layout == "local" else 80000
    c = Case(layout, [(L, 2), (9000, rows)], 8, 1, dtype or "bf16", window=L if layout == "local" else 0, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("layout,dtype", [("local", "bf16"), ("local", "e4m3"), ("folded", "bf16"), ("full", "bf16"),
                                          ("folded_e4m3", "")])
@pytest.mark.parametrize("rows", [2, 4, 8, 10])
def test_sharp_logits(layout, dtype, rows):
    """Logits of standard deviation 30: references rise and rows are rescaled."""
    c = Case(layout, at_most([(600, 10), (1500, 3)], rows), 8, 1, dtype or "bf16",
             window=1500 if layout == "local" else 0, seed=8, q_sigma=30.0)
    c.run()
    assert int(c.status.item()) == 0
    for b in range(2):
        want, size = c.want(b)
        got = c.out[c.cu[b]:c.cu[b + 1]].float().cpu().double().numpy()
        # the logits' own float32 error, 2^-24 of sums of |q k| up to 30 * 512 / sqrt(dim), a few tens of
        # additions deep, moves weights by 1e-3 at most; q's two terms on e4m3 pools by 2^-17 of its largest
        assert np.all(np.abs(got - want) <= (2.0 ** -8 * 3 + 4e-3) * size + 1e-6)


@pytest.mark.parametrize("layout,dtype", [("local", "e4m3"), ("folded_e4m3", ""), ("local", "bf16"), ("folded", "bf16")])
@pytest.mark.parametrize("n", [2, 4, 8, 9])
def test_long_tail(layout, dtype, n):
    """One token 2^11.5 above each of 1100 others: their weights together are a third of its own, and one
    by one below the smallest e4m3 number."""
    L = 1100
    c = Case(layout, [(L, n)], 8, 1, dtype or "bf16", window=L if layout == "local" else 0, seed=4, sigma=0.5)
    first = c.cells.float()
    # K: one direction, 2 for token 100 and 0 elsewhere, so that its logit is 8 (base e) and theirs 0
    page, off = int(c.table[0, 100 // 16]), 100 % 16
    x = first.clone()
    if layout == "local":
        x[:, :, 0] = 0
        x[page, :, 0, off, 7] = 2.0
    elif layout == "folded":
        x[:, :, 16:] = 0  # every dim of K but V[0:128)
        x[page, off // 8, 64, off % 8, 7] = 2.0
    else:
        x[:, :, 8:] = 0
        x[page, off // 8, 32, off % 8, 7] = 2.0
    x = torch.where(torch.isnan(first), first, x).to(c.cells.dtype)
    c.cells.view(torch.uint8).copy_(x.view(torch.uint8))
    c.q.zero_()
    c.q[:, :, 7] = 64.0 if layout == "local" else 4.0 * 512 ** 0.5
    c.run()
    c.check()


def test_decode_rows_agree():
    """One row with its own bit is a decode row."""
    for layout, kv, window in (("local", 4, 50), ("folded", 1, 0)):
        c = Case(layout, [(100, 1), (37, 1), (900, 1)], 8, kv, window=window, seed=2)
        got = c.run().float()
        out = torch.empty_like(c.q)
        ws = gw.alloc_workspace(c.pool, 8, 3, c.table.shape[1], 1, window or 1)
        d = c.dev
        if layout == "local":
            gw.decode_attn_local(c.pool, c.q, out, d["cu"], d["lens"], d["table"], ws, window)
        else:
            gw.decode_attn_global(c.pool, c.q, out, d["cu"], d["lens"], d["table"], ws)
        assert (got - out.float()).norm() <= 2.0 ** -7 * out.float().norm()


@pytest.mark.parametrize("plan", [[(700, 6), (1300, 17), (90, 33)], [(700, 6), (1300, 8), (90, 1)], [(700, 3), (1300, 4), (90, 1)]])
@pytest.mark.parametrize("layout,kv,window", [("local", 2, 300), ("folded", 1, 0), ("folded_e4m3", 1, 0)])
def test_rows_do_not_depend_on_the_batch(layout, kv, window, plan):
    c = Case(layout, plan, 8, kv, window=window, seed=6)
    most = max(n for _, n in plan)
    whole = c.run().clone()
    for cap in (1, 7, 0):
        gw.set_max_ctas(cap)
        try:
            assert torch.equal(c.run(max_q_rows=64 if most > 8 else most), whole)
        finally:
            gw.set_max_ctas(0)
    for b in range(3):
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        q, out = c.q[rows].contiguous(), torch.empty_like(c.q[rows])
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        n = plan[b][1]
        table = i32(c.table[b:b + 1].tolist())
        ws = gw.alloc_workspace_tree(c.pool, 8, 1, table.shape[1], most, window or 1)
        mask = torch.from_numpy(c.mask[rows]).cuda()
        if layout == "local":
            gw.tree_attn_local(c.pool, q, out, i32([0, n]), i32([plan[b][0]]), table, mask, i32(c.pos[rows].tolist()),
                               ws, window, max_q_rows=most)
        else:
            gw.tree_attn_global(c.pool, q, out, i32([0, n]), i32([plan[b][0]]), table, mask, ws, max_q_rows=most)
        assert torch.equal(out, whole[rows])


@pytest.mark.parametrize("layout,kv,window", [("local", 2, 64), ("folded", 1, 0), ("full", 1, 0), ("folded_e4m3", 1, 0)])
@pytest.mark.parametrize("few", [False, True])
def test_bad_metadata(layout, kv, window, few):
    """Sequences that are refused get zeros, pages out of range count as zeros; the others are as ever."""
    heads = 8 if not few else kv
    if few and layout != "local":
        return bad_few(layout)
    c = Case(layout, [(100, 6), (40, 8), (200, 5), (30, 3)], heads, kv, window=window, seed=9)
    good = c.run().clone()
    c.check()
    lens = c.lens.copy()
    lens[1] = 7  # below its rows
    lens[3] = c.table.shape[1] * 16 + 1
    out = c.run(lens=torch.from_numpy(lens).cuda())
    assert int(c.status.item()) == gw.GW_DEV_LEN_RANGE
    assert torch.equal(out[:6], good[:6]) and torch.equal(out[14:19], good[14:19])
    assert (out[6:14] == 0).all() and (out[19:] == 0).all()
    out = c.run(max_q_rows=6)
    assert int(c.status.item()) == gw.GW_DEV_LEN_RANGE
    assert (out[6:14] == 0).all() and torch.equal(out[14:], good[14:])
    table = c.table.copy()
    table[2, 11] = c.pages
    out = c.run(table=torch.from_numpy(table).cuda())
    assert int(c.status.item()) == gw.GW_DEV_PAGE_RANGE
    assert torch.equal(out[:14], good[:14]) and torch.equal(out[19:], good[19:])
    assert torch.isfinite(out[14:19]).all()
    if layout == "local":
        pos = c.pos.copy()
        pos[15] = 194  # before the drafts
        out = c.run(pos=torch.from_numpy(pos).cuda())
        assert int(c.status.item()) == gw.GW_DEV_POS_RANGE
        assert (out[15] == 0).all() and torch.equal(out[:14], good[:14])


def bad_few(layout):
    c = Case(layout, [(100, 3), (40, 4), (600, 2), (30, 1)], 8, seed=9)
    good = c.run().clone()
    c.check()
    lens, table = c.lens.copy(), c.table.copy()
    lens[1], lens[3], table[2, 20] = 3, c.table.shape[1] * 16 + 1, -1
    out = c.run(lens=torch.from_numpy(lens).cuda(), table=torch.from_numpy(table).cuda())
    assert int(c.status.item()) == gw.GW_DEV_LEN_RANGE | gw.GW_DEV_PAGE_RANGE
    assert torch.equal(out[:3], good[:3]) and (out[3:7] == 0).all() and (out[9:] == 0).all()
    assert torch.isfinite(out[7:9]).all() and not torch.equal(out[7:9], good[7:9])


def test_max_batch_and_idle_slots():
    plan = [((b * 37) % 150 + 5, b % 4) for b in range(256)]
    for layout, kv, window in (("local", 1, 40), ("folded", 1, 0)):
        c = Case(layout, plan, 8, kv, window=window, seed=12)
        for most in (3, 8, 20):  # few rows and many
            c.run(max_q_rows=most)
            c.check()


@pytest.mark.parametrize("layout,dtype", [("local", "bf16"), ("folded", "bf16")])
def test_pages_behind_4_gib(layout, dtype):
    """A sequence in the last pages of a pool of more than 2^32 bytes."""
    kv = 16 if layout == "local" else 1
    pages = (1 << 32) // (262144 if layout == "local" else 20480) + 20
    c = Case(layout, [(150, 9)], 32, kv, window=100 if layout == "local" else 0, seed=1)
    small, cells = c.pool, c.cells
    c.pool = gw.KVPool(layout, dtype, pages, kv)
    c.cells = c.pool.data.view(torch.bfloat16).view((pages,) + cells.shape[1:])
    c.cells[pages - cells.shape[0]:] = cells
    c.table = np.where((c.table >= 0) & (c.table < 1 << 20), c.table + pages - cells.shape[0], c.table).astype(np.int32)
    c.run()
    c.check()
    assert small.num_pages == cells.shape[0]


def test_graphs_share_a_workspace_and_streams():
    """Two captured calls of different shape on one workspace, replayed in turn with new inputs; a call on
    another stream."""
    a = Case("folded", [(700, 6), (1300, 12)], 8, seed=21)
    b = Case("folded", [(2000, 16)], 8, seed=22)
    want_a, want_b = a.run().clone(), b.run().clone()
    ws = a.ws if a.ws.numel() > b.ws.numel() else b.ws
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    graphs = []
    side = torch.cuda.Stream()
    for c in (a, b):
        c.run(ws=ws, status=status)
        torch.cuda.synchronize()
        out = torch.zeros_like(c.q)
        dev, most = c.dev, max(n for _, n in c.plan)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gw.tree_attn_global(c.pool, c.q, out, dev["cu"], dev["lens"], dev["table"], dev["mask"], ws, max_q_rows=most,
                                dev_status=status)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), want in zip(graphs, (want_a, want_b)):
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
    # the same graph over a shorter step: lengths and words are inputs
    a.dev["lens"].copy_(torch.tensor([6, 700], dtype=torch.int32))
    graphs[0][0].replay()
    a.plan, a.lens = [(6, 6), (700, 12)], np.array([6, 700], np.int32)
    a.out, a.status = graphs[0][1], status
    a.check()
    side.wait_stream(torch.cuda.default_stream())
    out, d = torch.full_like(b.q, float("nan")), b.dev
    side.wait_stream(torch.cuda.current_stream())
    gw.tree_attn_global(b.pool, b.q, out, d["cu"], d["lens"], d["table"], d["mask"], ws, max_q_rows=16, stream=side)
    side.synchronize()
    assert torch.equal(out, want_b)


def test_binding_refuses():
    c = Case("local", [(40, 4)], 8, 4, window=32, seed=1)
    c.run()
    d = c.dev
    args = [c.pool, c.q, c.out, d["cu"], d["lens"], d["table"], d["mask"], d["pos"], c.ws, 32]
    for at, bad in ((1, c.q.float()), (1, c.q[:, :, :128]), (2, c.out[:2]), (3, d["cu"][:1]), (3, d["cu"].long()),
                    (5, d["table"].t()), (6, d["mask"].int()), (6, d["mask"][:2]), (7, d["pos"][:3]), (6, d["mask"].cpu()),
                    (8, c.ws.cpu())):
        call = list(args)
        call[at] = bad
        with pytest.raises(gw.GwError):
            gw.tree_attn_local(*call, max_q_rows=4)
    with pytest.raises(gw.GwError, match="workspace_bytes"):
        gw.tree_attn_local(*args[:5], torch.zeros(1, 512, dtype=torch.int32, device="cuda"), *args[6:8], c.ws, 1 << 20)
