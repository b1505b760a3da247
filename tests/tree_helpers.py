"""Test-side glue for drafted trees: pools of random rows, trees, and attention,
norms, acceptance and moves by their definitions in float64 on the CPU."""

import math

import numpy as np
import torch

from paged_hybrid_attention_gb300 import gw

PAGE = 16
ROW = {"folded": (640, 8), "full": (1024, 8), "folded_e4m3": (640, 16)}


def kind_of(layout, dtype="bf16"):
    return torch.float8_e4m3fn if dtype == "e4m3" or layout == "folded_e4m3" else torch.bfloat16


def shape_of(layout, pages, kv_heads=1):
    if layout == "local":
        return (pages, kv_heads, 2, PAGE, 256)
    row, blk = ROW[layout]
    return (pages, 2, row // blk, 8, blk)


def new_pool(layout, pages, kv_heads=1, dtype="bf16", fill=0):
    """A pool and its rows as a typed tensor over the same memory."""
    dtype = "e4m3" if layout == "folded_e4m3" else dtype
    pool = gw.KVPool(layout, dtype, pages, kv_heads)
    pool.data.fill_(fill)
    return pool, pool.data.view(kind_of(layout, dtype)).view(shape_of(layout, pages, kv_heads))


def to64(x):
    return (x.float() if x.dtype != torch.float64 else x).double().cpu().numpy()


def kv_rows(cells, layout, table, tokens):
    """K and V [heads, tokens, dim], float64, of the tokens behind a block-table row."""
    t = np.asarray(tokens)
    page, off = np.asarray(table)[t // PAGE], t % PAGE
    x = to64(cells.view(torch.uint8)[torch.from_numpy(page).long().to(cells.device)].view(cells.dtype))
    if layout == "local":
        x = x[np.arange(len(t)), :, :, off]
        return x[:, :, 0].transpose(1, 0, 2), x[:, :, 1].transpose(1, 0, 2)
    x = x[np.arange(len(t)), off // 8, :, off % 8].reshape(len(t), -1)
    if layout == "full":
        return x[None, :, :512], x[None, :, 512:]
    return np.concatenate([x[:, 512:], x[:, 128:512]], 1)[None], x[None, :, :512]


def tree_of(rng, n):
    """Parents of n rows: chains that branch now and then."""
    return [-1] + [int(rng.choice([i - 1, i - 1, rng.integers(i)])) for i in range(1, n)]


def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def seen_by_tree(parent):
    """Row i's visible drafts: itself and its ancestors."""
    n = len(parent)
    m = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            m[i, j] = True
            j = parent[j]
    return m


def words(m):
    """A visibility matrix's rows as signed 64-bit words."""
    out = []
    for row in m:
        w = sum(1 << int(i) for i in np.nonzero(row)[0])
        out.append(w - (1 << 64) if w >> 63 else w)
    return out


def attend(q, k, v, sees, scale):
    """Rows q [n, heads, dim] over K, V [kv heads, tokens, dim] where sees [n,
    tokens]; and the sum of p |v|, which the tolerances count."""
    n, hq, dim = q.shape
    group = hq // k.shape[0]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(hq):
        kk, vv = k[h // group], v[h // group]
        for r in range(n):
            t = np.nonzero(sees[r])[0]
            if len(t) == 0:
                continue
            e = kk[t] @ q[r, h] * scale
            p = np.exp(e - e.max())
            p /= p.sum()
            out[r, h], size[r, h] = p @ vv[t], p @ np.abs(vv[t])
    return out, size


class Case:
    """A batch of trees over a pool of random rows.  `plan`: (length, rows) of
    each sequence; sees: "tree", or "any" for random words, some of them empty."""

    def __init__(self, layout, plan, heads, kv_heads=1, dtype="bf16", window=0, sees="tree", seed=0, spare=2,
                 sigma=1.0, q_sigma=1.0, extra_pages=0):
        rng = np.random.default_rng(seed)
        self.layout, self.plan, self.heads, self.window = layout, plan, heads, window
        self.dim = 256 if layout == "local" else 512
        self.scale = 1 / math.sqrt(self.dim)
        need = [-(-L // PAGE) for L, _ in plan]
        self.pages = sum(need) + 3
        self.pool, self.cells = new_pool(layout, self.pages, kv_heads, dtype, fill=0xff)  # NaN wherever no token is
        perm = rng.permutation(self.pages)
        self.table = np.full((len(plan), max(need + [1]) + spare), -7, np.int32)
        at = 0
        g = torch.Generator().manual_seed(seed)
        for b, (L, n) in enumerate(plan):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            lo = max(0, L - n - window + 1) if window else 0
            if lo > 0:
                self.table[b, :lo // PAGE] = 1 << 30  # pages behind the window: anything
            t = np.arange(lo, L)
            if len(t) == 0:
                continue
            page = torch.from_numpy(self.table[b, t // PAGE].astype(np.int64)).cuda()
            off = torch.from_numpy(t % PAGE).cuda()
            kind = self.cells.dtype
            if layout == "local":
                x = (torch.randn(len(t), kv_heads, 2, 256, generator=g) * sigma).to(kind).cuda()
                self.cells.view(torch.uint8 if kind != torch.bfloat16 else kind)[page, :, :, off] = \
                    x if kind == torch.bfloat16 else x.view(torch.uint8)
            else:
                row, blk = ROW[layout]
                x = (torch.randn(len(t), row // blk, blk, generator=g) * sigma).to(kind).cuda()
                self.cells.view(torch.uint8 if kind != torch.bfloat16 else kind)[page, off // 8, :, off % 8] = \
                    x if kind == torch.bfloat16 else x.view(torch.uint8)
        self.rows = sum(n for _, n in plan)
        self.q = (torch.randn(self.rows, heads, self.dim, generator=g) * q_sigma).to(torch.bfloat16).cuda()
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in plan])]).astype(np.int32)
        self.lens = np.array([L for L, _ in plan], np.int32)
        self.trees = [tree_of(rng, n) if n else [] for _, n in plan]
        self.sees = [seen_by_tree(t) if sees == "tree" else
                     (rng.random((len(t), len(t))) < rng.choice([0.0, 0.3, 1.0], size=(len(t), 1))) for t in self.trees]
        self.pos = np.array([L - n + d for (L, n), t in zip(plan, self.trees) for d in depths(t)], np.int32)
        self.mask = np.array([w for m in self.sees for w in words(m)], np.int64)

    def run(self, out=None, stream=None, max_q_rows=None, ws=None, status=None, mask=None, **other):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        self.out = torch.full_like(self.q, float("nan")) if out is None else out
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
        most = max([n for _, n in self.plan] + [1]) if max_q_rows is None else max_q_rows
        d = dict(cu=i32(self.cu), lens=i32(self.lens), table=i32(self.table), pos=i32(self.pos),
                 mask=torch.from_numpy(self.mask).cuda())
        d.update(other)
        self.dev = d
        self.ws = gw.alloc_workspace_tree(self.pool, self.heads, len(self.plan), self.table.shape[1], most,
                                          self.window or 1) if ws is None else ws
        if self.layout == "local":
            gw.tree_attn_local(self.pool, self.q, self.out, d["cu"], d["lens"], d["table"], d["mask"], d["pos"],
                               self.ws, self.window, max_q_rows=most, dev_status=self.status, stream=stream)
        else:
            gw.tree_attn_global(self.pool, self.q, self.out, d["cu"], d["lens"], d["table"], d["mask"], self.ws,
                                max_q_rows=most, dev_status=self.status, stream=stream)
        return self.out

    def want(self, b):
        """Sequence b's rows and their sum of p |v|."""
        L, n = self.plan[b]
        base, pos = L - n, self.pos[self.cu[b]:self.cu[b + 1]].astype(np.int64)
        lo = max(0, base - self.window + 1) if self.window else 0
        t = np.arange(lo, L)
        sees = np.concatenate([np.ones((n, base - lo), bool), self.sees[b]], 1)
        if self.window:
            at = np.concatenate([np.arange(lo, base), pos])
            sees &= at[None] > pos[:, None] - self.window
        k, v = kv_rows(self.cells, self.layout, self.table[b], t)
        return attend(to64(self.q[self.cu[b]:self.cu[b + 1]]), k, v, sees, self.scale)

    def check(self, status=0):
        """Every row within what its roundings allow: the weights' one rounding
        for the product, in numerator and denominator (2^-8 of a weight each),
        and the output's (2^-8), with float32 sums and logits beside them."""
        assert int(self.status.item()) == status, int(self.status.item())
        got = to64(self.out)
        for b in range(len(self.plan)):
            if self.plan[b][1] == 0:
                continue
            want, size = self.want(b)
            g = got[self.cu[b]:self.cu[b + 1]]
            assert np.isfinite(g).all(), b
            tol = 2.0 ** -8 * (2 * size + np.abs(want)) * 1.05 + 1e-6
            bad = np.abs(g - want) > tol
            assert not bad.any(), (b, self.plan[b], int(bad.sum()), float((np.abs(g - want) / tol).max()))
            assert (g[size.sum(-1) == 0] == 0).all()  # rows that see nothing
