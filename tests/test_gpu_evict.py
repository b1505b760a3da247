"""gw_kv_evict_select and gw_kv_evict_compact against plain loops on the host,
and an eviction as a decode loop uses it.  Choices and moved bytes are exact."""

import math

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G
from tests.test_gpu_acc import Cache

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- select
def _choose(w, L, budget, sinks, recent):
    """The kept indices by sorting, in Python."""
    if L <= budget:
        return list(range(L))
    mid = range(sinks, L - recent)
    rank = sorted(mid, key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
    return sorted([*range(sinks), *rank[:budget - sinks - recent], *range(L - recent, L)])


def _select(acc, lens, budget, sinks, recent, stream=None):
    keep = torch.full((len(lens), budget + 3), -9, dtype=torch.int32, device="cuda")
    n = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.kv_evict_select(acc, G.i32(lens), budget, keep, n, sinks, recent, status, stream)
    return keep, n, status


def _check_select(acc, lens, budget, sinks, recent):
    keep, n, status = _select(acc, lens, budget, sinks, recent)
    w = acc.cpu().double().numpy()
    keep, n = keep.cpu().numpy(), n.cpu().numpy()
    assert int(status) == 0
    for b, L in enumerate(lens):
        want = _choose(w[b].tolist(), L, budget, sinks, recent)
        assert n[b] == len(want)
        assert np.array_equal(keep[b, :n[b]], want), b
        assert np.all(keep[b, n[b]:] == -9)


def _weights(kind, batch, width, seed=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, width, generator=g)
    if kind == "tail":
        w = torch.exp(2 * x - 6)
    elif kind == "ties":
        w = torch.randint(0, 3, (batch, width), generator=g).float() / 4
    elif kind == "zeros":
        w = torch.where(x > 2, x, torch.zeros_like(x)) * torch.where(x < 0, -1.0, 1.0)     # 0 and -0
    elif kind == "close":                                                                  # neighbours in the last bits
        w = torch.full_like(x, 1.0).view(torch.int32).add(torch.randint(0, 7, x.shape, generator=g).int()).view(
            torch.float32)
    elif kind == "signs":
        w = x * 10.0 ** torch.randint(-38, 38, x.shape, generator=g).float()
    else:                                                                                  # odd: NaN, infinities
        w = x.clone()
        r = torch.rand(batch, width, generator=g)
        w[r < 0.2] = float("nan")
        w[(r >= 0.2) & (r < 0.4)] = float("inf")
        w[(r >= 0.4) & (r < 0.6)] = float("-inf")
        w.view(torch.int32)[(r >= 0.6) & (r < 0.7)] = -1                                   # NaN with the sign set
    return w.cuda()


@pytest.mark.parametrize("kind", ["tail", "ties", "zeros", "close", "signs", "odd"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 4, 16), (64, 0, 0), (100, 50, 50),
                                                 (1000, 3, 5), (1025, 0, 1024)])
def test_select_matches_sorting(kind, budget, sinks, recent):
    lens = [0, 1, 2, 39, 40, 41, 63, 64, 65, 100, 101, 999, 1000, 1001, 1024, 1025, 1026, 2047, 2500, 4099]
    _check_select(_weights(kind, len(lens), 4099), lens, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["tail", "ties", "close"])
def test_select_long(kind):
    for lens, budget in (([131072, 70001, 20000], 32768), ([300007], 5), ([16384, 16385, 131071], 16384)):
        _check_select(_weights(kind, len(lens), max(lens) + 1), lens, budget, 2, 3)


def test_select_very_long():
    """More tokens than any on-chip buffer of a sequence holds."""
    w = _weights("tail", 1, 1100003)
    _check_select(w, [1100003], 200000, 16, 4096)


@pytest.mark.parametrize("batch", [1, 2, 7, 40, 300])
def test_select_batches_and_row_strides(batch):
    """Odd row strides (no row but the first is aligned), many sequences;
    each row's choice is its own."""
    lens = [(b * 37) % 700 for b in range(batch)]
    room = _weights("tail", batch, 801)
    _check_select(room[:, :701], lens, 64, 2, 7)


def test_select_bad_lengths():
    acc = _weights("tail", 4, 100)
    keep, n, status = _select(acc, [50, -1, 101, 100], 10, 1, 1)
    assert int(status) == gw.GW_DEV_LEN_RANGE
    assert n.tolist() == [10, 0, 0, 10]
    assert bool((keep[1:3] == -9).all())
    w = acc.cpu().double().numpy()
    assert keep[0, :10].tolist() == _choose(w[0].tolist(), 50, 10, 1, 1)
    assert keep[3, :10].tolist() == _choose(w[3].tolist(), 100, 10, 1, 1)


# ------------------------------------------------------------------ compact
def _keep_of(g, L, n):
    return sorted(torch.randperm(L, generator=g)[:n].tolist())


def _moved(c, before, b, keep, dst_table):
    """The pool's rows of sequence b after the move, by plain indexing."""
    row, blk = {"folded": (80, 16), "full": (128, 16), "folded_e4m3": (40, 16)}[c.layout]
    src = before.view(-1, 2, row, 8, blk)
    out = []
    for j in keep:
        out.append(src[int(c.table[b, j // 16]), j % 16 // 8, :, j % 8])
    return torch.stack(out) if out else src[:0, 0, :, 0]


def _rows_at(c, b, table, tokens):
    row, blk = {"folded": (80, 16), "full": (128, 16), "folded_e4m3": (40, 16)}[c.layout]
    pool = c.pool.data.cpu().view(-1, 2, row, 8, blk)
    return torch.stack([pool[int(table[b, i // 16]), i % 16 // 8, :, i % 8] for i in tokens]) if tokens else pool[:0, 0, :, 0]


def _keep_tensor(keeps, width, fill=-5):
    t = torch.full((len(keeps), width), fill, dtype=torch.int32)
    for b, k in enumerate(keeps):
        t[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    return t.cuda()


LAYOUTS = ["folded", "full", "folded_e4m3"]
LENS = [0, 1, 16, 17, 100, 255, 256, 257, 300, 600, 1500]


def _choices(lens, seed=4):
    g = torch.Generator().manual_seed(seed)
    keeps = []
    for b, L in enumerate(lens):
        n = [L, 0, L // 2, max(0, L - 1), min(L, 7)][b % 5]
        keeps.append(_keep_of(g, L, n))
    return keeps


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", ["mixed", "tail", "every", "second", "last"])
def test_compact_in_place(layout, shape):
    """Random choices, the last tokens only, all, every second one, one: the
    moved rows byte for byte, everything else of the pool as it was."""
    c = Cache(layout, LENS, 8)
    keeps = {"mixed": _choices(LENS), "tail": [list(range(L - L // 3, L)) for L in LENS],
             "every": [list(range(L)) for L in LENS], "second": [list(range(1, L, 2)) for L in LENS],
             "last": [[L - 1] if L else [] for L in LENS]}[shape]
    before = c.pool.data.cpu().clone()
    acc = torch.rand(len(LENS), c.width * 16 + 3, device="cuda")
    old = acc.clone()
    gw.kv_evict_compact(c.pool, c.bt, c.n, _keep_tensor(keeps, 1600), G.i32([len(k) for k in keeps]), acc,
                        dev_status=c.status)
    assert int(c.status) == 0
    expect = before.clone().view(-1, 2, {"folded": 80, "full": 128, "folded_e4m3": 40}[layout], 8, 16)
    for b, (L, keep) in enumerate(zip(LENS, keeps)):
        rows = _moved(c, before, b, keep, c.table)
        for i in range(len(keep)):
            expect[int(c.table[b, i // 16]), i % 16 // 8, :, i % 8] = rows[i]
        m = len(keep)
        assert torch.equal(acc[b, :m], old[b, torch.tensor(keep, dtype=torch.long, device="cuda")])
        assert bool((acc[b, m:L] == 0).all()) and torch.equal(acc[b, L:], old[b, L:])
    assert torch.equal(c.pool.data.cpu(), expect.reshape(-1))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_compact_into_other_pages(layout):
    """Into pages of their own, shared prefix pages left behind or kept in
    place (the same page in both tables)."""
    lens = [300, 40, 513]
    c = Cache(layout, lens, 8)
    keeps = _choices([300, 40, 513], 9)
    keeps[0] = list(range(32)) + keeps[0][40:]           # the first two pages stay whole
    held = set(c.table[c.table >= 0].tolist())
    grown = gw.KVPool(layout, c.pool.dtype, c.pool.num_pages + 120)
    grown.data[:c.pool.nbytes].copy_(c.pool.data)
    before = grown.data.cpu().clone()
    c.pool = grown
    dst = torch.arange(3 * 40, dtype=torch.int32).view(3, 40) + (grown.num_pages - 120)
    dst[0, :2] = c.table[0, :2]
    acc = torch.rand(3, c.width * 16, device="cuda")
    gw.kv_evict_compact(grown, c.bt, c.n, _keep_tensor(keeps, 600), G.i32([len(k) for k in keeps]), None,
                        dst.cuda(), c.status)
    assert int(c.status) == 0
    for b, keep in enumerate(keeps):
        assert torch.equal(_rows_at(c, b, dst, list(range(len(keep)))), _moved(c, before, b, keep, dst))
    page = grown.page_bytes
    after = grown.data.cpu()
    for p in held:                                       # what was read is as it was
        assert torch.equal(after[p * page:(p + 1) * page], before[p * page:(p + 1) * page])


def test_compact_refuses_bad_values():
    lens = [100, 100, 100, 100, 100, 100]
    c = Cache("folded", lens, 8)
    before = c.pool.data.cpu().clone()
    keeps = [[0, 5, 5, 9], [3, 2, 50], [7, 100], [-1, 4], [1, 2, 3], [10, 20]]
    keep_lens = [4, 3, 2, 2, 101, 2]
    c.n[5] = 10 ** 6
    acc = torch.rand(6, c.width * 16, device="cuda")
    old = acc.clone()
    gw.kv_evict_compact(c.pool, c.bt, c.n, _keep_tensor(keeps, 120), G.i32(keep_lens), acc, dev_status=c.status)
    assert int(c.status) == gw.GW_DEV_KEEP_RANGE | gw.GW_DEV_LEN_RANGE
    good = {0: {1: 5, 3: 9}, 1: {0: 3, 2: 50}, 2: {0: 7}, 3: {1: 4}, 4: {}, 5: {}}
    expect = before.clone().view(-1, 2, 80, 8, 16)
    src = before.view(-1, 2, 80, 8, 16)
    want = old.clone()
    for b, moves in good.items():
        for i, j in moves.items():
            expect[int(c.table[b, i // 16]), i % 16 // 8, :, i % 8] = src[int(c.table[b, j // 16]), j % 16 // 8, :, j % 8]
            want[b, i] = old[b, j]
        if b < 4:
            want[b, keep_lens[b]:100] = 0
    assert torch.equal(c.pool.data.cpu(), expect.reshape(-1))
    assert torch.equal(acc, want)
    # pages out of range: those rows stay, the others move
    c = Cache("folded", [64], 8)
    before = c.pool.data.cpu().clone()
    c.bt[0, 3] = c.pool.num_pages
    gw.kv_evict_compact(c.pool, c.bt, c.n, _keep_tensor([[20, 50, 33]], 3)[:, :2], G.i32([2]), dev_status=c.status)
    assert int(c.status) == gw.GW_DEV_PAGE_RANGE
    expect = before.clone().view(-1, 2, 80, 8, 16)
    expect[int(c.table[0, 0]), 0, :, 0] = before.view(-1, 2, 80, 8, 16)[int(c.table[0, 1]), 0, :, 4]
    assert torch.equal(c.pool.data.cpu(), expect.reshape(-1))
    # more kept tokens than the other table has pages
    c.status.zero_()
    mid = c.pool.data.cpu().clone()
    gw.kv_evict_compact(c.pool, c.bt, c.n, _keep_tensor([list(range(40))], 40), G.i32([40]), None,
                        torch.zeros(1, 2, dtype=torch.int32, device="cuda"), c.status)
    assert int(c.status) == gw.GW_DEV_KEEP_RANGE and torch.equal(c.pool.data.cpu(), mid)


def test_largest_batches():
    """65535 sequences, the most that a call takes."""
    batch = 65535
    acc = _weights("tail", batch, 9)
    lens = torch.arange(batch, dtype=torch.int32, device="cuda") % 10
    keep = torch.full((batch, 4), -9, dtype=torch.int32, device="cuda")
    n = torch.zeros(batch, dtype=torch.int32, device="cuda")
    gw.kv_evict_select(acc, lens, 4, keep, n, 1, 1)
    assert torch.equal(n, lens.clamp(max=4))
    w, k = acc.cpu().double().numpy(), keep.cpu().numpy()
    for b in [*range(0, 40), *range(batch - 40, batch)]:
        L = b % 10
        assert k[b, :min(L, 4)].tolist() == _choose(w[b].tolist(), L, 4, 1, 1)
    pool = gw.KVPool("folded_e4m3", "e4m3", batch)
    rows = pool.data.view(batch, 2, 40, 8, 16)
    rows.copy_(torch.arange(16, dtype=torch.uint8, device="cuda").view(2, 1, 8, 1).expand(2, 40, 8, 16))
    table = torch.arange(batch, dtype=torch.int32, device="cuda").flip(0).view(batch, 1).contiguous()
    wide = torch.zeros(batch, 16, device="cuda")
    wide[:, :9] = acc
    gw.kv_evict_compact(pool, table, lens, keep, n, wide)
    got = rows[table[:, 0].long()][:, 0, 7, :4, 3].int()        # the token that lies in each of the first four places
    place = torch.arange(4, device="cuda")
    assert torch.equal(got, torch.where(place < n[:, None], keep, place.int()))
    want, every = torch.zeros(batch, 16, device="cuda"), torch.arange(16, device="cuda")
    want[:, :9] = torch.where(every[:9] < lens[:, None], want[:, :9], acc)         # behind the end: as it was
    want[:, :4] = torch.where(place < n[:, None], acc.gather(1, keep.clamp(min=0).long()), want[:, :4])
    assert torch.equal(wide, want)


def test_binding_refuses():
    c = Cache("folded", [20], 8)
    keep, n = _keep_tensor([[1, 2]], 4), G.i32([2])
    with pytest.raises(gw.GwError, match="kv_evict_select"):
        gw.kv_evict_select(torch.rand(1, 20, device="cuda"), c.n, 5, keep, n)
    with pytest.raises(gw.GwError, match="kv_evict_select"):
        gw.kv_evict_select(torch.rand(1, 20, device="cuda").half(), c.n, 2, keep, n)
    with pytest.raises(gw.GwError, match="kv_evict_select"):
        gw.kv_evict_select(torch.rand(2, 30, device="cuda")[:, 9:], G.i32([3, 3]), 2, torch.stack([keep[0]] * 2),
                           G.i32([0, 0]))
    with pytest.raises(gw.GwError, match="kv_evict_compact"):
        gw.kv_evict_compact(c.pool, c.bt, c.n, keep, n, torch.zeros(1, 31, device="cuda"))
    with pytest.raises(gw.GwError, match="kv_evict_compact"):
        gw.kv_evict_compact(c.pool, c.bt, c.n, keep.long(), n)
    local = gw.KVPool("local", "bf16", 2, 1)
    with pytest.raises(gw.GwError, match="window"):
        gw.kv_evict_compact(local, c.bt, c.n, keep, n)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_early_inputs_behind_a_cut(layout):
    """Choice, move and the next attention over the new lengths without a
    kernel between them, with the index inputs read early: the same bits."""
    lens = [3000, 40, 700, 1, 260]
    c = Cache(layout, lens, 16)
    start, q = c.pool.data.clone(), c.q.cuda()
    got = []
    try:
        for early in (False, True, True):
            c.pool.data.copy_(start)
            acc, keep = c.new_acc(), torch.full((5, 256), -1, dtype=torch.int32, device="cuda")
            n, out = torch.zeros(5, dtype=torch.int32, device="cuda"), [torch.empty_like(q) for _ in range(3)]
            torch.cuda.synchronize()
            gw.set_early_inputs(early)
            c.run(acc, q=q, out=out[0], lse=None)
            gw.kv_evict_select(acc, c.n, 256, keep, n, 2, 30, c.status)
            gw.kv_evict_compact(c.pool, c.bt, c.n, keep, n, acc, dev_status=c.status)
            gw.decode_attn_global_acc(c.pool, q, out[1], None, acc, c.cu, n, c.bt, c.ws, dev_status=c.status)
            gw.decode_attn_global(c.pool, q, out[2], c.cu, n, c.bt, c.ws, dev_status=c.status)
            torch.cuda.synchronize()
            got.append([t.view(torch.uint8).clone() for t in (*out, acc, keep, n, c.pool.data)])
    finally:
        gw.set_early_inputs(False)
    assert int(c.status) == 0
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_two_streams_at_once():
    """Calls on two streams, each with its own cache, weights and workspace,
    overlap without changing either's results."""
    lens = [5000, 300, 2100]
    jobs = []
    for k in range(2):
        c = Cache(LAYOUTS[k], lens, 8, seed=20 + k)
        jobs.append(dict(c=c, start=c.pool.data.clone(), acc=c.new_acc(), q=c.q.cuda(), stream=torch.cuda.Stream(),
                         keep=torch.full((3, 512), -1, dtype=torch.int32, device="cuda"),
                         n=torch.zeros(3, dtype=torch.int32, device="cuda"), got=[]))
        jobs[-1]["out"] = torch.empty_like(jobs[-1]["q"])

    def go(j, stream):
        c = j["c"]
        c.run(j["acc"], q=j["q"], out=j["out"], lse=None, stream=stream)
        gw.kv_evict_select(j["acc"], c.n, 512, j["keep"], j["n"], 3, 64, c.status, stream)
        gw.kv_evict_compact(c.pool, c.bt, c.n, j["keep"], j["n"], j["acc"], dev_status=c.status, stream=stream)

    for turn in range(3):
        for j in jobs:
            j["c"].pool.data.copy_(j["start"])
            j["acc"].zero_()
        torch.cuda.synchronize()
        for j in jobs:
            go(j, j["stream"] if turn else None)
            if not turn:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for j in jobs:
            assert int(j["c"].status) == 0
            j["got"].append([t.clone() for t in (j["out"], j["acc"], j["keep"], j["n"], j["c"].pool.data)])
    for j in jobs:
        for turn in (1, 2):
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(j["got"][turn], j["got"][0]))


# ------------------------------------------------------- a decode loop with both
@pytest.mark.parametrize("layout", LAYOUTS)
def test_decode_loop_with_eviction(layout):
    """Steps of append, q rotation, attention with weights, and a cut: the
    cache's attention after the cut is attention over the kept tokens'
    rows, whose choice follows from the weights added up before; captured in
    a graph, the same bits."""
    heads, lens, budget = 8, [90, 200, 33], 48
    c = Cache(layout, lens, heads, width=16)
    table = gw.rope_cs_scaled(1e6, 128, 512, 400, kind="ramp", factor=4.0, orig_max_pos=100)
    g = torch.Generator(device="cuda").manual_seed(8)
    free = torch.arange(c.pool.num_pages, c.pool.num_pages + 3 * 16, dtype=torch.int32, device="cuda").view(3, 16)
    grown = gw.KVPool(layout, c.pool.dtype, c.pool.num_pages + 48)
    grown.data[:c.pool.nbytes].copy_(c.pool.data)
    c.pool, c.bt = grown, torch.where(c.bt >= 0, c.bt, free)
    start = grown.data.clone()
    acc = c.new_acc()
    keep = torch.full((3, budget), -1, dtype=torch.int32, device="cuda")
    keep_lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    pos, n = G.i32(lens), G.i32(lens)
    steps = [(torch.randn(3, heads, 512, generator=g, device="cuda").to(torch.bfloat16),
              torch.randn(3, 512, generator=g, device="cuda").to(torch.bfloat16)) for _ in range(4)]
    outs = [torch.zeros(3, heads, 512, dtype=torch.bfloat16, device="cuda") for _ in steps]
    seqs = torch.arange(3, device="cuda")
    trace = []

    def loop(note=None):
        c.pool.data.copy_(start)
        acc.zero_()
        pos.copy_(G.i32(lens) if note is not None else first)
        n.copy_(pos)
        for t, (q, k) in enumerate(steps):
            slot = c.bt[seqs, (n // 16).long()] * 16 + n % 16
            gw.kv_append(c.pool, k, k, slot, pos, table, c.status)
            n.add_(1)
            qr = gw.rope_rows(q, pos, table, rot_dim=128)
            pos.add_(1)
            c.n = n
            gw.decode_attn_global_acc(c.pool, qr, outs[t], None, acc, c.cu, n, c.bt, c.ws, dev_status=c.status)
            if note is not None:
                note(t, qr)
            if t == 1:
                gw.kv_evict_select(acc, n, budget, keep, keep_lens, 2, 8, c.status)
                gw.kv_evict_compact(c.pool, c.bt, n, keep, keep_lens, acc, dev_status=c.status)
                n.copy_(keep_lens)

    first = G.i32(lens)

    def rows(b, count):
        row, blk, kind = {"folded": (640, 8, torch.bfloat16), "full": (1024, 8, torch.bfloat16),
                          "folded_e4m3": (640, 16, torch.float8_e4m3fn)}[layout]
        i = torch.arange(count, device="cuda")
        x = c.pool.data.view(kind).float().view(-1, 2, row // blk, 8, blk)[c.bt[b, i // 16].long(), i % 16 // 8, :, i % 8]
        return x.reshape(count, row).double().cpu()

    def note(t, qr):
        state = dict(q=qr.double().cpu(), out=outs[t].clone(), acc=acc.clone(), n=n.tolist(),
                     rows=[rows(b, int(n[b])) for b in range(3)])
        trace.append(state)

    loop(note)
    assert int(c.status) == 0
    total = [torch.zeros(0, dtype=torch.float64) for _ in lens]
    for t, s in enumerate(trace):
        for b in range(3):
            x, m = s["rows"][b], s["n"][b]
            if t == 2:                                   # the cut: follow the library's choice, check it below
                idx = keep[b, :int(keep_lens[b])].cpu().long()
                before = trace[1]["rows"][b]
                assert torch.equal(x[:-1], before[idx])
                w = trace[1]["acc"][b].double().cpu().tolist()
                assert idx.tolist() == _choose(w, trace[1]["n"][b], budget, 2, 8)
                total[b] = total[b][idx]
            k = x[:, :512] if layout == "full" else torch.cat([x[:, 512:], x[:, 128:512]], 1)
            v = x[:, 512:] if layout == "full" else x[:, :512]
            p = torch.softmax(s["q"][b] @ k.T / math.sqrt(512), -1)
            mx, rl = G.errors(G.to_f64(s["out"][b]), (p @ v).numpy())
            assert mx <= G.MAX_ABS and rl <= G.REL_L2
            total[b] = torch.cat([total[b], torch.zeros(m - len(total[b]), dtype=torch.float64)]) + p.sum(0)
            # logits here are below 8 and sum |q k| below 32: the bound of the weights' tests
            assert bool(((s["acc"][b, :m].double().cpu() - total[b]).abs() <= (2.0 ** -11 + 2.0 ** -17) * total[b]).all())
    final = [o.clone() for o in outs]
    bytes_after, acc_after, n_after = c.pool.data.clone(), acc.clone(), n.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        loop()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for _ in range(2):
        keep.fill_(-1)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, final))
    assert torch.equal(c.pool.data, bytes_after) and torch.equal(acc, acc_after) and torch.equal(n, n_after)
