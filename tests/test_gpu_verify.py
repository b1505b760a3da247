"""Verification steps as a program runs them, captured in a graph: norms, rotation
and append of every draft, attention of the trees, the accepted path and its move,
over a local and a global layer; against caches that hold the accepted tokens only."""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import PAGE, depths, kv_rows, new_pool, seen_by_tree, tree_of, words

pytestmark = pytest.mark.gpu
VOCAB, HEADS, KV, WINDOW, MAX_POS = 24, 8, 4, 40, 512


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Layer:
    """A layer whose projections are a function of the token."""

    def __init__(self, layout, dtype, pages, g):
        self.local = layout == "local"
        self.dim, rot = (256, 256) if self.local else (512, 128)
        self.kv = KV if self.local else 1
        heads = HEADS + (2 * KV if self.local else 1)
        self.proj = torch.randn(VOCAB, heads, self.dim, generator=g, device="cuda", dtype=torch.bfloat16)
        self.qw = 1 + 0.2 * torch.randn(self.dim, generator=g, device="cuda")
        self.kw = 1 + 0.2 * torch.randn(self.dim, generator=g, device="cuda")
        self.cs = gw.rope_cs(1e4 if self.local else 1e6, rot, self.dim, MAX_POS)
        self.layout = layout
        self.pool, self.cells = new_pool(layout, pages, self.kv, dtype)
        self.clean, self.clean_cells = new_pool(layout, pages, self.kv, dtype)

    def append(self, pool, tokens, slot, pos, out):
        x = self.proj[tokens.long()]
        k = x[:, HEADS:HEADS + self.kv]
        v = x[:, HEADS + self.kv:] if self.local else k
        gw.norm_rope_append(pool, x[:, :HEADS], k, v, self.qw, self.kw, slot, pos, self.cs, out)


@pytest.mark.parametrize("dtype,layout,n", [("bf16", "folded", 4), ("bf16", "full", 16), ("e4m3", "folded_e4m3", 9),
                                            ("bf16", "folded", 40)])
def test_steps(dtype, layout, n):
    rng = np.random.default_rng(n)
    g = torch.Generator(device="cuda").manual_seed(n)
    batch, width = 3, 16
    pages = batch * width
    table_np = rng.permutation(pages).reshape(batch, width)
    table = i32(table_np)
    layers = [Layer("local", dtype, pages, g), Layer(layout, "e4m3" if layout == "folded_e4m3" else "bf16", pages, g)]
    # the newest token of each is not cached yet
    tokens = [[int(t) for t in rng.integers(0, VOCAB, m + 1)] for m in (0, 13, 100)]
    for b, have in enumerate(tokens):
        at = np.arange(len(have) - 1)
        for x in layers if len(at) else ():
            for pool in (x.pool, x.clean):
                x.append(pool, i32(have[:-1]), i32(table_np[b, at // PAGE] * PAGE + at % PAGE), i32(at),
                         torch.empty(len(at), HEADS, x.dim, dtype=torch.bfloat16, device="cuda"))
    rows = batch * n
    zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    d = dict(draft=zeros(rows), target=zeros(rows), parent=zeros(rows), slot=zeros(rows), pos=zeros(rows),
             lens=zeros(batch), path=zeros(batch, n), path_lens=zeros(batch), next=zeros(batch), new_lens=zeros(batch),
             mask=torch.zeros(rows, dtype=torch.int64, device="cuda"))
    cu, status = i32(np.arange(batch + 1) * n), zeros(1)
    for x in layers:
        x.q = torch.empty(rows, HEADS, x.dim, dtype=torch.bfloat16, device="cuda")
        x.out = torch.empty_like(x.q)
        x.ws = gw.alloc_workspace_tree(x.pool, HEADS, batch, width, n, WINDOW)

    def step():
        for x in layers:
            x.append(x.pool, d["draft"], d["slot"], d["pos"], x.q)
            if x.local:
                gw.tree_attn_local(x.pool, x.q, x.out, cu, d["lens"], table, d["mask"], d["pos"], x.ws, WINDOW,
                                   max_q_rows=n, dev_status=status)
            else:
                gw.tree_attn_global(x.pool, x.q, x.out, cu, d["lens"], table, d["mask"], x.ws, max_q_rows=n,
                                    dev_status=status)
        gw.tree_accept(cu, d["lens"], d["parent"], d["draft"], d["target"], d["path"], d["path_lens"], d["next"],
                       d["new_lens"], dev_status=status)
        for x in layers:
            gw.kv_tree_move([x.pool], cu, d["lens"], table, d["path"], d["path_lens"], dev_status=status)

    graph = None
    for k in range(6):
        host = {name: [] for name in ("draft", "target", "parent", "slot", "pos", "lens", "mask")}
        want_paths = []
        for b in range(batch):
            base = len(tokens[b]) - 1
            tree = tree_of(rng, n)
            draft = [tokens[b][-1]] + [int(t) for t in rng.integers(0, VOCAB, n - 1)]
            # what the target chooses: often one of the row's children's drafts
            target = []
            for i in range(n):
                kids = [j for j in range(n) if tree[j] == i]
                target.append(draft[kids[int(rng.integers(len(kids)))]] if kids and rng.random() < 0.8 else
                              int(rng.integers(VOCAB)))
            path = [0]
            while True:
                kids = [j for j in range(1, n) if tree[j] == path[-1] and draft[j] == target[path[-1]]]
                if not kids:
                    break
                path.append(kids[0])
            want_paths.append((path, target[path[-1]], draft))
            at = base + np.arange(n)
            host["draft"] += draft
            host["target"] += target
            host["parent"] += tree
            host["slot"] += list(table_np[b, at // PAGE] * PAGE + at % PAGE)
            host["pos"] += [base + x for x in depths(tree)]
            host["lens"].append(base + n)
            host["mask"] += words(seen_by_tree(tree))
        for name, v in host.items():
            d[name].copy_(torch.tensor(np.array(v)))
        if graph is None:
            step()  # once in the open, then captured
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            saved = [x.pool.data.clone() for x in layers]
            with torch.cuda.graph(graph):
                step()
            for x, s in zip(layers, saved):
                x.pool.data.copy_(s)
            # the step has run: its drafts again, over a cache whose rows have moved
        graph.replay()
        assert int(status.item()) == 0
        for b, (path, last, draft) in enumerate(want_paths):
            m = int(d["path_lens"][b])
            assert d["path"][b, :m].tolist() == path and int(d["next"][b]) == last
            assert int(d["new_lens"][b]) == host["lens"][b] - n + m
            first = len(tokens[b]) - 1
            # the same tokens one after the other into a clean cache
            ids = [draft[i] for i in path]
            pos = np.arange(first, first + m)
            for x in layers:
                q = torch.empty(m, HEADS, x.dim, dtype=torch.bfloat16, device="cuda")
                x.append(x.clean, i32(ids), i32(table_np[b, pos // PAGE] * PAGE + pos % PAGE), i32(pos), q)
                at = torch.tensor([b * n + i for i in path], device="cuda")
                assert torch.equal(x.q[at], q)
                # each accepted row's attention is the decode row's over the clean cache
                got, want = x.out[at].float(), torch.empty_like(q)
                w = gw.alloc_workspace(x.clean, HEADS, m, width, 1, WINDOW)
                rows_of = table[b:b + 1].expand(m, width).contiguous()
                if x.local:
                    gw.decode_attn_local(x.clean, q, want, i32(np.arange(m + 1)), i32(pos + 1), rows_of, w, WINDOW)
                else:
                    gw.decode_attn_global(x.clean, q, want, i32(np.arange(m + 1)), i32(pos + 1), rows_of, w)
                # both round weights for the product and the row: 2^-8 each, in norm well below 2^-6
                assert (got - want.float()).norm() <= 2.0 ** -6 * want.float().norm()
            tokens[b] += ids[1:] + [last]
    # wherever a token has been committed the caches hold the same rows
    for x in layers:
        for b in range(batch):
            for a, c in zip(kv_rows(x.cells, x.layout, table_np[b], range(len(tokens[b]) - 1)),
                            kv_rows(x.clean_cells, x.layout, table_np[b], range(len(tokens[b]) - 1))):
                assert np.array_equal(a, c)
    assert len(tokens[0]) > 7 and len(tokens[2]) > 107
