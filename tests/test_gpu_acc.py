"""gw_decode_attn_global_acc against attention in float64 over the cached rows.

Tolerances.  A logit is a sum of 512 exact products of stored values in
float32, scaled once: with 2^-24 a step and the tensor cores' sums truncated
(2^-23 a step, 32 steps of 16 products), it is off by at most 2^-17 of
scale * sum |q k|.  A weight e^(logit - lse) is then off, relatively, by
twice that (its own and the normaliser's logit), by the base-2 scaling of
logits up to a few tens (2^-23 * 2 * |logit|) and by exp2 and the sums
(below 2^-18 for sums of up to 2^17 terms added pairwise and in tiles).
lse is off by the same, absolutely.  Outputs keep the attention tolerance of
the other tests.
"""

import math

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

ROW = {"folded": (640, 8), "full": (1024, 8), "folded_e4m3": (640, 16)}


class Cache:
    """A pool of random rows held by sequences of these lengths in scattered
    pages; what no sequence holds is NaN."""

    def __init__(self, layout, lens, heads, seed=1, width=None, spread=1.0, rows=None):
        g = torch.Generator().manual_seed(seed)
        self.layout, self.lens, self.heads = layout, lens, heads
        row, blk = ROW[layout]
        need = [(max(n, 0) + 15) // 16 for n in lens]
        self.width = width or max(max(need), 1)
        n_pages = sum(need) + 3
        perm = torch.randperm(n_pages, generator=g)
        data = torch.randn(n_pages, 16, row, generator=g) * spread
        kind = torch.float8_e4m3fn if layout == "folded_e4m3" else torch.bfloat16
        data = data.to(torch.bfloat16).to(kind)
        self.table = torch.full((len(lens), self.width), -7, dtype=torch.int32)
        used = torch.zeros(n_pages, 16, dtype=torch.bool)
        at = 0
        values = data.float()
        self.tokens = []
        for b, n in enumerate(lens):
            p = perm[at:at + need[b]]
            at += need[b]
            m = min(need[b], self.width)
            self.table[b, :m] = p[:m].int()
            t = torch.arange(max(n, 0))
            used[p[t // 16], t % 16] = True
            self.tokens.append(values[p].reshape(-1, row)[:max(n, 0)].double())
        raw = data.view(torch.uint8) if kind != torch.bfloat16 else data.view(torch.int16)
        raw[~used] = 0x7f if kind != torch.bfloat16 else 0x7fc0                 # NaN
        raw = raw.view(n_pages, 2, 8, row // blk, blk).permute(0, 1, 3, 2, 4).contiguous()
        self.pool = gw.KVPool(layout, "e4m3" if kind != torch.bfloat16 else "bf16", n_pages)
        self.pool.data.copy_(raw.view(torch.uint8).view(-1).cuda())
        self.rows = rows if rows is not None else [1] * len(lens)
        self.q = torch.randn(sum(self.rows), heads, 512, generator=g).to(torch.bfloat16)
        cu = [0]
        for r in self.rows:
            cu.append(cu[-1] + r)
        self.cu, self.n = G.i32(cu), G.i32(lens)
        self.bt = self.table.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = gw.alloc_workspace_acc(self.pool, heads, len(lens), self.width)

    def kv(self, b):
        x = self.tokens[b]
        if self.layout == "full":
            return x[:, :512], x[:, 512:]
        return torch.cat([x[:, 512:], x[:, 128:512]], 1), x[:, :512]

    def new_acc(self, fill=0.0, extra=0):
        return torch.full((len(self.lens), self.width * 16 + extra), fill, device="cuda")

    def run(self, acc, decay=1.0, lse=True, q=None, scale=None, stream=None, out=None):
        q = self.q.cuda() if q is None else q
        out = torch.full_like(q, float("nan")) if out is None else out
        lse = torch.full(q.shape[:2], float("nan"), device="cuda") if lse is True else lse
        gw.decode_attn_global_acc(self.pool, q, out, lse, acc, self.cu, self.n, self.bt, self.ws, decay, scale,
                                  self.status, stream)
        return out, lse

    def want(self, b, scale=None):
        """(rows, lse, weights summed over the heads, their tolerance) in float64."""
        scale = 1 / math.sqrt(512) if scale is None else scale
        k, v = self.kv(b)
        q = self.q[int(self.cu[b])].double()
        e = q @ k.T * scale
        lse = torch.logsumexp(e, -1)
        w = torch.exp(e - lse[:, None])
        size = q.abs() @ k.T.abs() * scale
        rel = 2 * 2.0 ** -17 * size.max() + 2.0 ** -22 * e.abs().max() + 2.0 ** -18
        return w @ v, lse, w.sum(0), float(rel)

    def check(self, out, lse, acc, old=None, decay=1.0, scale=None, before=None):
        for b, n in enumerate(self.lens):
            if n < 1 or self.rows[b] != 1:
                continue
            r = int(self.cu[b])
            rows, want_lse, w, rel = self.want(b, scale)
            mx, rl = G.errors(G.to_f64(out[r]), rows.numpy())
            assert mx <= G.MAX_ABS and rl <= G.REL_L2, (b, mx, rl)
            if lse is not None:
                assert float((lse[r].double().cpu() - want_lse).abs().max()) <= rel + 2.0 ** -22 * float(
                    want_lse.abs().max())
            base = 0.0 if not decay else decay * old[b, :n].double().cpu()
            total = base + w
            off = (acc[b, :n].double().cpu() - total).abs()
            assert bool((off <= rel * w + 2.0 ** -23 * total).all()), (b, float((off / total).max()), rel)


LAYOUTS = ["folded", "full", "folded_e4m3"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("heads", [8, 16, 32])
def test_lengths_at_the_edges(layout, heads):
    """One token, page, tile and chunk edges, several chunks; entries behind a
    sequence's end and another step's acc rows stay as they were."""
    c = Cache(layout, [1, 2, 15, 16, 17, 63, 64, 65, 511, 512, 513, 1100, 3000], heads)
    acc = torch.rand(len(c.lens), c.width * 16 + 5, device="cuda")
    old = acc.clone()
    out, lse = c.run(acc)
    assert int(c.status) == 0
    c.check(out, lse, acc, old)
    for b, n in enumerate(c.lens):
        assert torch.equal(acc[b, n:], old[b, n:])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_decay_and_sums_over_steps(layout):
    c = Cache(layout, [700, 40], 16)
    acc = c.new_acc(float("nan"))
    out, lse = c.run(acc, decay=0.0)                    # old values are not read
    c.check(out, lse, acc, decay=0.0)
    first = acc.clone()
    for b, n in enumerate(c.lens):
        assert bool(acc[b, n:].isnan().all())
        assert abs(float(acc[b, :n].double().sum()) - 16) < 1e-3
    c.run(acc, decay=0.5, lse=None)
    for b, n in enumerate(c.lens):
        want = 1.5 * first[b, :n].double()
        assert bool(((acc[b, :n].double() - want).abs() <= 2.0 ** -22 * want).all())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_peaked_and_large_logits(layout):
    """Logits of up to some hundreds: weights underflow to zero, the peak
    holds nearly all."""
    c = Cache(layout, [900, 33], 8, spread=4.0)
    acc = c.new_acc()
    out, lse = c.run(acc, scale=0.6)
    assert bool(acc.isfinite().all()) and float(acc.min()) >= 0
    for b, n in enumerate(c.lens):
        _, want_lse, w, rel = c.want(b, 0.6)
        off = (acc[b, :n].double().cpu() - w).abs()
        assert bool((off <= rel * w + 2.0 ** -100).all())
        assert float((lse[b].double().cpu() - want_lse).abs().max()) <= rel + 2.0 ** -22 * float(want_lse.abs().max())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_idle_slots_prompt_rows_and_bad_sequences(layout):
    """Slots without a row, with several rows, of length 0 or beyond the
    block table: their acc stays; the others' results do not change."""
    lens = [300, 50, 0, 200, -3, 128, 97]
    c = Cache(layout, lens, 8, rows=[1, 0, 0, 2, 1, 1, 1], width=19)
    c.n[5] = 19 * 16 + 1
    acc = c.new_acc(2.0)
    out, lse = c.run(acc)
    assert int(c.status) == gw.GW_DEV_LEN_RANGE
    for b in (1, 2, 3, 4, 5):
        assert bool((acc[b] == 2.0).all())
    c.rows = [1, 0, 0, 0, 0, 0, 1]
    c.check(out, lse, acc, torch.full_like(acc, 2.0))
    for b in (4, 5):                                     # invalid lengths: zero rows, no keys
        r = int(c.cu[b])
        assert bool((out[r] == 0).all()) and bool((lse[r] == float("-inf")).all())
    alone = Cache(layout, lens, 8, rows=[1, 0, 0, 2, 1, 1, 1], width=19)
    alone.n = G.i32([300, 0, 0, 0, 0, 0, 0])
    acc1 = alone.new_acc(2.0)
    out1, _ = alone.run(acc1)
    assert torch.equal(acc1[0], acc[0]) and torch.equal(out1[0], out[0])


def test_bad_pages_get_no_weight():
    c = Cache("folded", [100, 60], 8)
    c.bt[0, 2] = 10 ** 6
    c.bt[1] = -1
    acc = c.new_acc(1.0)
    out, lse = c.run(acc)
    assert int(c.status) == gw.GW_DEV_PAGE_RANGE
    w = acc[0, :100] - 1.0
    assert bool((w[32:48] == 0).all()) and abs(float(w.double().sum()) - 8) < 1e-3
    assert bool((acc[1] == 1.0).all()) and bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_same_rows_as_the_plain_call(layout):
    """The rows agree with gw_decode_attn_global's to a step of their
    rounding (the weights' sum is rounded differently), and do not depend on
    the batch; a long sequence in 64-bit offsets of a wide workspace."""
    c = Cache(layout, [5000, 31, 20000], 32)
    acc = c.new_acc()
    out, _ = c.run(acc)
    plain = torch.empty_like(out)
    ws = gw.alloc_workspace(c.pool, 32, 3, c.width, 1, 1)
    gw.decode_attn_global(c.pool, c.q.cuda(), plain, c.cu, c.n, c.bt, ws)
    mx, rl = G.errors(G.to_f64(out), G.to_f64(plain))
    assert mx <= G.MAX_ABS and rl <= G.REL_L2
    one = c.new_acc()
    full_n = c.n.clone()
    c.n = torch.where(torch.arange(3, device="cuda") == 2, full_n, torch.zeros_like(full_n)).to(torch.int32)
    out2, _ = c.run(one)
    assert torch.equal(one[2], acc[2]) and torch.equal(out2[2], out[2])
    again = c.new_acc()
    c.n = full_n
    out3, _ = c.run(again)
    assert torch.equal(again, acc) and torch.equal(out3, out)


def test_wide_workspace_offsets():
    """Logits beyond 2^31 elements into the workspace (a short sequence in
    the last of many wide slots)."""
    batch, width = 34, 131072
    c = Cache("folded", [20] + [0] * (batch - 2) + [777], 32, rows=[1] + [0] * (batch - 2) + [1], width=width)
    assert (batch - 1) * width * 16 * 32 > 2 ** 31
    acc = c.new_acc()
    out, lse = c.run(acc)
    assert int(c.status) == 0
    c.check(out, lse, acc, torch.zeros_like(acc))


def test_pages_beyond_4_gib():
    """Page offsets past 32 bits: the same rows at the end of a 6 GB pool."""
    c = Cache("folded", [900, 64, 1], 8)
    acc = c.new_acc()
    out, lse = c.run(acc)
    small = c.pool
    big = gw.KVPool("folded", "bf16", 300000)
    off = big.num_pages - small.num_pages
    assert off * big.page_bytes > 2 ** 32
    big.data[off * big.page_bytes:].copy_(small.data)
    c.pool, c.bt = big, torch.where(c.bt >= 0, c.bt + off, c.bt)
    acc2 = c.new_acc()
    out2, lse2 = c.run(acc2)
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and torch.equal(acc2, acc)
    keep = torch.arange(0, 900, 3, dtype=torch.int32, device="cuda").view(1, 300).repeat(3, 1)
    n = G.i32([300, 22, 1])
    before = big.data[off * big.page_bytes:].clone()
    for pool, table in ((small, c.bt - off), (big, c.bt)):
        gw.kv_evict_compact(pool, torch.where(c.bt >= 0, table, c.bt), c.n, keep, n, dev_status=c.status)
    assert int(c.status) == 0
    assert torch.equal(big.data[off * big.page_bytes:], small.data) and not torch.equal(before, small.data)


def test_largest_batch():
    """4096 sequences, the most that a call takes."""
    lens = [1 + b % 23 for b in range(4096)]
    c = Cache("folded", lens, 8)
    acc = c.new_acc()
    out, lse = c.run(acc)
    assert int(c.status) == 0
    some = [0, 1, 22, 23, 2047, 4000, 4094, 4095]
    c.rows = [1 if b in some else 0 for b in range(4096)]
    c.check(out, lse, acc, torch.zeros_like(acc))
    assert bool(((acc.double().sum(1) - 8).abs() < 1e-4).all())


def test_graph_streams_and_launch_settings():
    c = Cache("folded", [900, 64, 1], 16)
    acc = c.new_acc()
    out, lse = c.run(acc)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    acc2 = c.new_acc()
    torch.cuda.synchronize()
    out2, lse2 = c.run(acc2, stream=side, q=(q := c.q.cuda()), out=torch.empty_like(q),
                       lse=torch.empty_like(lse))
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and torch.equal(acc2, acc)
    # two graphs that share the workspace, replayed one after the other
    graphs = []
    for _ in range(2):
        a, o, l = c.new_acc(), torch.empty_like(out), torch.empty_like(lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(a, q=q, out=o, lse=l)
        graphs.append((graph, a, o, l))
    for _ in range(2):
        for graph, a, o, l in graphs:
            a.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, a, o, l in graphs:
            assert torch.equal(a, acc) and torch.equal(o, out) and torch.equal(l, lse)
    try:
        gw.set_early_inputs(True)
        gw.set_max_ctas(5)
        a = c.new_acc()
        o, l = c.run(a)
        assert torch.equal(a, acc) and torch.equal(o, out) and torch.equal(l, lse)
    finally:
        gw.set_early_inputs(False)
        gw.set_max_ctas(0)


def test_prompt_tail_as_batch_entries():
    """The last rows of a prompt as decode rows of several entries that share
    a block-table row, each with its own length."""
    c = Cache("folded", [200], 8)
    lens = [197, 198, 199, 200]
    c.lens, c.rows = lens, [1] * 4
    c.tokens = [c.tokens[0][:n] for n in lens]
    c.cu, c.n, c.bt = G.i32(range(5)), G.i32(lens), c.bt.repeat(4, 1)
    c.q = torch.randn(4, 8, 512, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    c.ws = gw.alloc_workspace_acc(c.pool, 8, 4, c.width)
    acc = c.new_acc()
    out, lse = c.run(acc)
    c.check(out, lse, acc, torch.zeros_like(acc))


def test_binding_refuses():
    c = Cache("folded", [20], 8)
    acc = c.new_acc()
    for bad in (acc.double(), acc[:, :16], acc.repeat(2, 1), acc.t()):
        with pytest.raises(gw.GwError, match="gw_decode_attn_global_acc"):
            c.run(bad)
    with pytest.raises(gw.GwError):
        c.run(acc.cpu())
    with pytest.raises(gw.GwError):
        c.run(acc, q=c.q.float().cuda())
    with pytest.raises(gw.GwError):
        c.run(acc, lse=torch.zeros(1, 9, device="cuda"))
