"""Operators that verify drafted tokens over the paged caches, with the cases
they are measured at.

A verification step gives each sequence up to 64 rows: the newest token and a
tree of drafts behind it.  Three operators take it through a layer: the norms
of q and k heads with their rotation and the append (`norm_append`), attention
of the tree's rows over the cache (`tree_local`, `tree_global`), and, once the
target has chosen its tokens, the accepted path and the move of its rows to
the front of the drafts' (`commit`).

With `own` false, `run` computes them in plain torch operations; with `own`
true it makes the library's calls.
"""

import math
import random

import torch

own = False

PAGE = 16
EPS = 1e-6
# layout of a global cache: elements of a token row, elements of a 16-byte block, type
GLOBAL = {
    "folded": (640, 8, torch.bfloat16),
    "full": (1024, 8, torch.bfloat16),
    "folded_e4m3": (640, 16, torch.float8_e4m3fn),
}
LOCAL = {"local": torch.bfloat16, "local_e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a local layer: 16 rows (latency)
        dict(name="norm_decode", op="norm_append", layout="local", rows=16, heads=32, kv_heads=16, packed=True,
             v_norm=True, max_pos=8192),
        # a tree step of a global layer: 16 sequences of 16 drafts
        dict(name="norm_tree", op="norm_append", layout="folded", rows=256, heads=32, kv_heads=1, packed=False,
             v_norm=True, max_pos=131072),
        # four 2048-token prompts of a local layer, from the packed projection, into the e4m3 cache
        dict(name="norm_prompt", op="norm_append", layout="local_e4m3", rows=8192, heads=32, kv_heads=16, packed=True,
             v_norm=False, max_pos=8192),
        # two short sequences, five drafts each, a small local layer (latency)
        dict(name="tree_local_small", op="tree_local", layout="local", heads=8, kv_heads=4, batch=2, idle=0,
             min_len=37, max_len=100, drafts=5, window=32, blind=False),
        # the serving step's sequences with 16 drafts each
        dict(name="tree_local_serving", op="tree_local", layout="local", heads=32, kv_heads=16, batch=16, idle=0,
             min_len=512, max_len=8192, drafts=16, window=1024, blind=False),
        # 64 sequences on the e4m3 cache, an odd number of drafts, some slots idle
        dict(name="tree_local_e4m3", op="tree_local", layout="local_e4m3", heads=32, kv_heads=16, batch=64, idle=3,
             min_len=4096, max_len=32768, drafts=7, window=1024, blind=False),
        # two short sequences of the full K and V control cache (latency)
        dict(name="tree_global_small", op="tree_global", layout="full", heads=8, kv_heads=1, batch=2, idle=0,
             min_len=37, max_len=100, drafts=5, window=0, blind=False),
        # the serving step's sequences with 16 drafts each
        dict(name="tree_global_serving", op="tree_global", layout="folded", heads=32, kv_heads=1, batch=16, idle=0,
             min_len=512, max_len=8192, drafts=16, window=0, blind=False),
        # long contexts: 8 sequences of 131072 tokens, four drafts each
        dict(name="tree_global_long", op="tree_global", layout="folded", heads=32, kv_heads=1, batch=8, idle=0,
             min_len=131072, max_len=131072, drafts=4, window=0, blind=False),
        # wide trees on the e4m3 cache
        dict(name="tree_global_wide", op="tree_global", layout="folded_e4m3", heads=16, kv_heads=1, batch=8, idle=0,
             min_len=16384, max_len=32768, drafts=33, window=0, blind=False),
        # two sequences, one global layer (latency)
        dict(name="commit_small", op="commit", layout="full", kv_heads=1, pools=1, batch=2, drafts=5, accept=3),
        # 16 sequences of 16 drafts, the 40 local layers of a 48-layer stack
        dict(name="commit_stack", op="commit", layout="local", kv_heads=16, pools=40, batch=16, drafts=16, accept=5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_append", "tree_local", "tree_local", "tree_global", "tree_global", "commit"])
    if op == "norm_append":
        layout = rng.choice(list(LOCAL) + list(GLOBAL))
        local = layout in LOCAL
        kv = rng.choice([1, 2, 4, 8, 16]) if local else 1
        heads = kv * rng.choice([1, 2, 3, 4, 8]) if local else rng.choice([8, 16, 32])
        return dict(op=op, layout=layout, rows=_log(rng, 1, 8192 * 32 // max(32, heads)), heads=heads, kv_heads=kv,
                    packed=rng.random() < 0.5, v_norm=rng.random() < 0.5 if local else True,
                    max_pos=_log(rng, 1, 131072))
    if op == "commit":
        layout = rng.choice(list(LOCAL) + list(GLOBAL))
        drafts = rng.choice([1, 2, 3, 5, 8, 16, 31, 64])
        return dict(op=op, layout=layout, kv_heads=rng.choice([1, 2, 4, 16]) if layout in LOCAL else 1,
                    pools=_log(rng, 1, 40), batch=_log(rng, 1, 32), drafts=drafts, accept=rng.randint(1, drafts))
    batch = _log(rng, 1, 64)
    drafts = _log(rng, 1, 64)
    idle = rng.randint(0, batch // 2)
    if op == "tree_local":
        kv = rng.choice([1, 2, 4, 8, 16])
        window = _log(rng, 1, 1024)
        max_len = _log(rng, drafts, 16384)
        return dict(op=op, layout=rng.choice(list(LOCAL)), heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv,
                    batch=batch, idle=idle, min_len=rng.randint(drafts, max_len), max_len=max_len, drafts=drafts,
                    window=window, blind=rng.random() < 0.3)
    heads = rng.choice([8, 16, 32])
    layout = rng.choice(list(GLOBAL))
    room = 8 * 131072 * 4 * 32 // (batch * drafts * heads)  # no more work than the longest listed case
    cached = (8 if layout != "full" else 5) * 131072 // batch
    max_len = _log(rng, drafts, max(drafts, min(131072, room, cached)))
    return dict(op=op, layout=layout, heads=heads, kv_heads=1, batch=batch, idle=idle,
                min_len=rng.randint(drafts, max_len), max_len=max_len, drafts=drafts, window=0,
                blind=rng.random() < 0.3)


# --------------------------------------------------------------- the inputs
def _lens(case):
    """The batch's lengths: spread evenly from min_len to max_len."""
    n = case["batch"] - case["idle"]
    lo, hi = case["min_len"], case["max_len"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(g, layout, kv_heads, pages):
    """Cached rows: local [page][kv head][K, V][16][256], global [page][2][column block][8][block]."""
    if layout in LOCAL:
        shape, kind = (pages, kv_heads, 2, PAGE, 256), LOCAL[layout]
    else:
        row, blk, kind = GLOBAL[layout]
        shape = (pages, 2, row // blk, 8, blk)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).to(kind)


def _table(g, need):
    """Block tables over scattered pages for sequences of need[b] pages, -1 behind their last."""
    total, width = sum(need), max(1, max(need))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = _i32([sum(need[:i]) for i in range(len(need))])[:, None]
    col = torch.arange(width, device="cuda")[None]
    at = (first + col).clamp(max=total - 1).long()
    return torch.where(col < _i32(need)[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _tree(rng, n):
    """Parents of n rows, row 0 the root: chains that branch now and then."""
    return [-1] + [rng.choice([i - 1, i - 1, rng.randrange(i)]) for i in range(1, n)]


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _mask(parent):
    """Each row's visible drafts, its ancestors and itself, as the bits of a signed 64-bit word."""
    m = []
    for i, p in enumerate(parent):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return [x - (1 << 64) if x >> 63 else x for x in m]


def _handle(case, pools):
    """What a program that uses the library keeps for its caches: the pool descriptors."""
    from paged_hybrid_attention_gb300 import gw
    e4m3 = case["layout"].endswith("e4m3")
    layout = "local" if case["layout"] in LOCAL else case["layout"]
    return [gw.KVPool(layout, "e4m3" if e4m3 else "bf16", p.shape[0], case["kv_heads"],
                      storage=p.view(torch.uint8).view(-1)) for p in pools]


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    s = dict(case=case)
    op, layout = case["op"], case["layout"]
    local = layout in LOCAL
    dim, rot, theta = (256, 256, 1e4) if local else (512, 128, 1e6)
    if op == "norm_append":
        rows, hq, kv = case["rows"], case["heads"], case["kv_heads"]
        size = [hq, kv, kv] if local else [hq, 1]
        if case["packed"]:
            x = torch.randn(rows, sum(size), dim, generator=g, device="cuda", dtype=torch.bfloat16)
            parts = list(x.split(size, 1))
        else:
            parts = [torch.randn(rows, n, dim, generator=g, device="cuda", dtype=torch.bfloat16) for n in size]
        s["q"], s["k"], s["v"] = parts[0], parts[1], parts[-1]  # global K and V come from one projection
        s["qw"] = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        s["kw"] = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        s["pool"] = _pool(g, layout, kv, (rows + PAGE - 1) // PAGE + 1)
        s["slot"] = torch.randperm(s["pool"].shape[0] * PAGE, generator=g, device="cuda")[:rows].to(torch.int32)
        s["pos"] = torch.randint(0, case["max_pos"], (rows,), generator=g, device="cuda", dtype=torch.int32)
        f = theta ** (torch.arange(rot // 2, device="cuda", dtype=torch.float64) * -2 / dim)
        a = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * f
        s["cs"] = torch.stack([a.cos(), a.sin()], -1).float()
        s["out"] = torch.empty(rows, hq, dim, dtype=torch.bfloat16, device="cuda")
        s["handle"] = _handle(case, [s["pool"]]) if own else None
        return s
    if op == "commit":
        n, batch = case["drafts"], case["batch"]
        base = [rng.randrange(0, 1024) for _ in range(batch)]
        parent, draft, target = [], [], []
        for _ in range(batch):
            # a path of `accept` rows whose drafts are what the target chose; every other row misses
            path = [0] + sorted(rng.sample(range(1, n), case["accept"] - 1))
            p, d, t = _tree(rng, n), [rng.randrange(1 << 17) * 2 for _ in range(n)], []
            for a, b in zip(path, path[1:]):
                p[b] = a
            t = [rng.randrange(1 << 17) * 2 + 1 for _ in range(n)]  # odd: no draft has it
            for a, b in zip(path, path[1:]):
                t[a] = d[b]
                for i in range(a + 1, b):
                    if p[i] == a and d[i] == d[b]:
                        d[i] += 2
            parent, draft, target = parent + p, draft + d, target + t
        s["parent"], s["draft"], s["target"] = _i32(parent), _i32(draft), _i32(target)
        s["base"] = base
        s["lens"] = _i32([b + n for b in base])
        s["cu"] = torch.arange(batch + 1, device="cuda", dtype=torch.int32) * n
        # the pages of the drafts; those before them are not touched
        first = [b // PAGE for b in base]
        need = [(b + n - 1) // PAGE + 1 - f for b, f in zip(base, first)]
        tail = _table(g, need)
        width = max(f + k for f, k in zip(first, need))
        s["table"] = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        for b in range(batch):
            s["table"][b, first[b]:first[b] + need[b]] = tail[b, :need[b]]
        pages = batch * ((n + PAGE - 2) // PAGE + 1)  # wherever the drafts begin in a page
        s["pools"] = [_pool(g, layout, case["kv_heads"], pages) for _ in range(case["pools"])]
        s["path"] = torch.full((batch, n), -1, dtype=torch.int32, device="cuda")
        for name in ("path_lens", "next", "new_lens"):
            s[name] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        s["handle"] = _handle(case, s["pools"]) if own else None
        return s
    lens = _lens(case)
    rng.shuffle(lens)
    live = len(lens)
    n, hq = case["drafts"], case["heads"]
    s["trees"] = [_tree(rng, n) for _ in lens]
    masks = [_mask(t) for t in s["trees"]]
    s["blind"] = []
    if case["blind"]:  # rows of a padded tree: they see no draft, not even themselves
        for b in range(live):
            i = rng.randrange(n)
            masks[b][i] = 0
            s["blind"].append(i)
    s["lens"] = _i32(lens + [0] * (case["batch"] - live))
    s["mask"] = torch.tensor([x for m in masks for x in m], dtype=torch.int64, device="cuda")
    s["pos"] = _i32([size - n + d for size, t in zip(lens, s["trees"]) for d in _depths(t)])
    s["cu"] = (torch.arange(case["batch"] + 1, device="cuda", dtype=torch.int32) * n).clamp(max=live * n)
    s["table"] = _table(g, [(x + PAGE - 1) // PAGE for x in lens] + [0] * (case["batch"] - live))
    s["pool"] = _pool(g, layout, case["kv_heads"], int((s["table"] >= 0).sum()))
    s["q"] = torch.randn(live * n, hq, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["host_lens"] = lens
    if own:
        from paged_hybrid_attention_gb300 import gw
        s["handle"] = _handle(case, [s["pool"]])
        s["ws"] = gw.alloc_workspace_tree(s["handle"][0], hq, case["batch"], s["table"].shape[1], n,
                                          case["window"] or 1)
    return s


# ------------------------------------------------------------------ one pass
def _turn(x, cs, rot):
    """The half pairs of x's first rot dims turned by cs [rows, 1, rot / 2, 2]."""
    x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
    c, t = cs[..., 0], cs[..., 1]
    return torch.cat([x0 * c - x1 * t, x1 * c + x0 * t, x[..., rot:]], -1)


def _norm_append(s):
    c = s["case"]
    local = c["layout"] in LOCAL
    rot = 256 if local else 128
    cs = s["cs"][s["pos"].long()][:, None]

    def unit(x):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)

    q = _turn(unit(s["q"]) * s["qw"], cs, rot)
    k = _turn(unit(s["k"]) * s["kw"], cs, rot)
    v = unit(s["v"]) if c["v_norm"] else s["v"].float()
    pool = s["pool"]
    kind = pool.dtype
    page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
    raw = pool.view(torch.uint8) if kind != torch.bfloat16 else pool

    def cell(x):
        x = x.to(kind)
        return x.view(torch.uint8) if kind != torch.bfloat16 else x

    if local:
        raw[page, :, 0, off], raw[page, :, 1, off] = cell(k), cell(v)
    else:
        if c["layout"] == "full":
            row = torch.cat([k, v], -1)
        else:
            row = torch.cat([v, k[..., :128]], -1)
            q = torch.cat([q[..., :128], q[..., 128:] * s["kw"][128:]], -1)
        blk = GLOBAL[c["layout"]][1]
        raw[page, off // 8, :, off % 8] = cell(row.view(row.shape[0], -1, blk))
    return q.to(torch.bfloat16), pool


def _tokens(s, b, first, last):
    """K and V [kv heads, tokens, dim] of tokens [first, last) of sequence b, in float32."""
    layout = s["case"]["layout"]
    p0, p1 = first // PAGE, (last - 1) // PAGE + 1
    pages = s["pool"].view(torch.uint8)[s["table"][b, p0:p1].long()].view(s["pool"].dtype).float()
    if layout in LOCAL:
        x = pages.permute(2, 1, 0, 3, 4).reshape(2, pages.shape[1], -1, 256)
        k, v = x[0], x[1]
    else:
        x = pages.permute(0, 1, 3, 2, 4).reshape(1, (p1 - p0) * PAGE, -1)
        v = x[..., 512:] if layout == "full" else x[..., :512]
        k = x[..., :512] if layout == "full" else torch.cat([x[..., 512:], x[..., 128:512]], -1)
    cut = slice(first - p0 * PAGE, last - p0 * PAGE)
    return k[:, cut], v[:, cut]


def _tree_attn(s):
    c = s["case"]
    n, hq, kv = c["drafts"], c["heads"], c["kv_heads"]
    dim = 256 if c["layout"] in LOCAL else 512
    out = s["out"]
    for b, size in enumerate(s["host_lens"]):
        base = size - n
        pos = s["pos"][b * n:(b + 1) * n].long()
        first = max(0, base - c["window"] + 1) if c["window"] else 0
        k, v = _tokens(s, b, first, size)
        at = torch.arange(first, size, device="cuda")
        bits = (s["mask"][b * n:(b + 1) * n, None] >> torch.arange(n, device="cuda")) & 1 == 1
        seen = torch.cat([torch.ones(n, base - first, dtype=torch.bool, device="cuda"), bits], 1)
        if c["window"]:
            at = torch.where(at < base, at, pos[(at - base).clamp(min=0)])
            seen &= at[None] > pos[:, None] - c["window"]
        q = s["q"][b * n:(b + 1) * n].float().view(n, kv, hq // kv, dim).permute(1, 2, 0, 3)
        e = q.reshape(kv, -1, dim) @ k.transpose(1, 2) * (1 / math.sqrt(dim))
        e = e.view(kv, hq // kv, n, -1).masked_fill(~seen, -math.inf)
        top = e.amax(-1, keepdim=True)
        w = torch.exp(e - torch.where(top.isinf(), torch.zeros_like(top), top))
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
        o = (w.view(kv, -1, w.shape[-1]) @ v).view(kv, hq // kv, n, dim)
        out[b * n:(b + 1) * n] = o.permute(2, 0, 1, 3).reshape(n, hq, dim).to(torch.bfloat16)
    return out


def _commit(s):
    c = s["case"]
    n, batch = c["drafts"], c["batch"]
    parent, draft, target = (s[x].view(batch, n).long() for x in ("parent", "draft", "target"))
    col = torch.arange(n, device="cuda")[None]
    at = torch.zeros(batch, 1, dtype=torch.long, device="cuda")
    walking = torch.ones(batch, 1, dtype=torch.bool, device="cuda")
    path, steps = s["path"], torch.zeros(batch, 1, dtype=torch.long, device="cuda")
    for i in range(n):
        path[:, i:i + 1] = torch.where(walking, at.int(), path[:, i:i + 1])
        steps += walking
        hit = (parent == at) & (draft == target.gather(1, at)) & (col > 0)
        found = hit.any(1, keepdim=True)
        at = torch.where(walking & found, hit.int().argmax(1, keepdim=True), at)
        walking = walking & found
    s["path_lens"].copy_(steps[:, 0])
    s["next"].copy_(target.gather(1, at)[:, 0])
    base = s["lens"] - n
    s["new_lens"].copy_(base + steps[:, 0])
    b, i = (col < steps).nonzero(as_tuple=True)
    to, src = base[b] + i, base[b] + path[b, i]
    tp, sp = s["table"][b, to // PAGE].long(), s["table"][b, src // PAGE].long()
    to, src = (to % PAGE).long(), (src % PAGE).long()
    for pool in s["pools"]:
        raw = pool.view(torch.uint8)
        if c["layout"] in LOCAL:
            raw[tp, :, :, to] = raw[sp, :, :, src]
        else:
            raw[tp, to // 8, :, to % 8] = raw[sp, src // 8, :, src % 8]
    return [path, s["path_lens"], s["next"], s["new_lens"]] + s["pools"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm_append": _norm_append, "tree_local": _tree_attn, "tree_global": _tree_attn,
                "commit": _commit}[op](s)
    from paged_hybrid_attention_gb300 import gw
    if op == "norm_append":
        gw.norm_rope_append(s["handle"][0], s["q"], s["k"], s["v"], s["qw"], s["kw"], s["slot"], s["pos"], s["cs"],
                            s["out"], eps=EPS, v_norm=c["v_norm"])
        return s["out"], s["pool"]
    if op == "tree_local":
        gw.tree_attn_local(s["handle"][0], s["q"], s["out"], s["cu"], s["lens"], s["table"], s["mask"], s["pos"],
                           s["ws"], c["window"], max_q_rows=c["drafts"])
        return s["out"]
    if op == "tree_global":
        gw.tree_attn_global(s["handle"][0], s["q"], s["out"], s["cu"], s["lens"], s["table"], s["mask"], s["ws"],
                            max_q_rows=c["drafts"])
        return s["out"]
    gw.tree_accept(s["cu"], s["lens"], s["parent"], s["draft"], s["target"], s["path"], s["path_lens"], s["next"],
                   s["new_lens"])
    gw.kv_tree_move(s["handle"], s["cu"], s["lens"], s["table"], s["path"], s["path_lens"])
    return [s["path"], s["path_lens"], s["next"], s["new_lens"]] + s["pools"]


# ------------------------------------------------------------- what it takes
def _row_bytes(case):
    """Bytes that one token has in the cache."""
    if case["layout"] in LOCAL:
        return case["kv_heads"] * 512 * (1 if case["layout"] == "local_e4m3" else 2)
    row, _, kind = GLOBAL[case["layout"]]
    return row * (2 if kind == torch.bfloat16 else 1)


def work(case):
    op = case["op"]
    local = case["layout"] in LOCAL
    dim = 256 if local else 512
    if op == "norm_append":
        rows, hq, kv = case["rows"], case["heads"], case["kv_heads"]
        values = hq + (2 * kv if local else 1)
        rot = 256 if local else 128
        moved = rows * (values * dim * 2 + hq * dim * 2 + _row_bytes(case))
        return {"bytes": moved + min(rows, case["max_pos"]) * rot * 4 + 8 * rows, "flops": rows * values * dim * 6}
    if op == "commit":
        moved = case["batch"] * (case["accept"] - 1)
        rows = case["batch"] * case["drafts"]
        return {"bytes": moved * 2 * _row_bytes(case) * case["pools"] + 12 * rows + 4 * (moved + 4 * case["batch"]),
                "flops": rows}
    lens = _lens(case)
    n, hq = case["drafts"], case["heads"]
    seen = [min(x, case["window"] - 1 + n) if case["window"] else x for x in lens]
    rows = len(lens) * n
    return {"bytes": sum(seen) * _row_bytes(case) + rows * (hq * dim * 4 + 12),
            "flops": sum(seen) * n * hq * 4 * dim}


# ----------------------------------------------- the definitions, in 64 bits
def _exact_norm(s):
    c = s["case"]
    local = c["layout"] in LOCAL
    half = 128 if local else 64
    cs = s["cs"].double()[s["pos"].long()]
    turn = torch.complex(cs[..., 0], cs[..., 1])

    def head(x, w):  # one head of every row
        x = x.double()
        y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
        if w is None:
            return y
        y = y * w.double()
        z = torch.complex(y[:, :half], y[:, half:2 * half]) * turn
        y[:, :half], y[:, half:2 * half] = z.real, z.imag
        return y

    q = torch.stack([head(s["q"][:, h], s["qw"]) for h in range(c["heads"])], 1)
    if c["layout"].startswith("folded"):
        q[..., 128:] *= s["kw"].double()[128:]
    pool = s["pool"].double() if s["pool"].dtype == torch.bfloat16 else s["pool"].float().double()
    page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
    for h in range(c["kv_heads"]):
        k = head(s["k"][:, h], s["kw"])
        v = head(s["v"][:, h], None) if c["v_norm"] else s["v"][:, h].double()
        if local:
            pool[page, h, 0, off], pool[page, h, 1, off] = k, v
            continue
        row = torch.cat([k, v], -1) if c["layout"] == "full" else torch.cat([v, k[:, :128]], -1)
        blk = GLOBAL[c["layout"]][1]
        for e in range(0, row.shape[1], blk):
            pool[page, off // 8, e // blk, off % 8] = row[:, e:e + blk]
    return q, pool


def _exact_tree(s):
    """Row by row of the tree: its tokens are the cached ones and its ancestors, by their walk to the root."""
    c = s["case"]
    n, hq, kv, w = c["drafts"], c["heads"], c["kv_heads"], c["window"]
    local = c["layout"] in LOCAL
    dim = 256 if local else 512
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, size in enumerate(s["host_lens"]):
        base = size - n
        t = torch.arange(max(0, base - w + 1) if w else 0, size, device="cuda")
        page = s["table"][b].long()[t // PAGE]
        pool = s["pool"] if s["pool"].dtype == torch.bfloat16 else s["pool"].float()
        tree, depth = s["trees"][b], _depths(s["trees"][b])
        allowed = torch.zeros(n, len(t), dtype=torch.bool)
        place = t.cpu()
        for i in range(n):
            here = base + depth[i]
            sees = (place < base) & ((place > here - w) if w else torch.ones_like(place, dtype=torch.bool))
            walk = -1 if c["blind"] and s["blind"][b] == i else i
            while walk >= 0:
                # a blind row is still its descendants' ancestor
                if not w or base + depth[walk] > here - w:
                    sees[base + walk - int(place[0])] = True
                walk = tree[walk]
            allowed[i] = sees
        allowed = allowed.cuda()
        for h in range(kv):
            if local:
                k, v = pool[page, h, 0, t % PAGE].double(), pool[page, h, 1, t % PAGE].double()
            else:
                x = pool[page, t % PAGE // 8, :, t % 8].reshape(len(t), -1).double()
                v = x[:, 512:] if c["layout"] == "full" else x[:, :512]
                k = x[:, :512].clone()
                if c["layout"] != "full":
                    k[:, :128] = x[:, 512:]
            group = hq // kv
            for g in range(h * group, (h + 1) * group):
                e = s["q"][b * n:(b + 1) * n, g].double() @ k.T / math.sqrt(dim)
                e[~allowed] = -math.inf
                lse = torch.logsumexp(e, -1, keepdim=True)
                p = torch.where(allowed, torch.exp(e - lse), torch.zeros_like(e))
                out[b * n:(b + 1) * n, g] = p @ v
    return out


def _exact_commit(s):
    """The whole numbers have no rounding; the pools by one accepted row after the other."""
    c = s["case"]
    n, table = c["drafts"], s["table"].tolist()
    parent, draft, target = (s[x].tolist() for x in ("parent", "draft", "target"))
    pools = [p.double() if p.dtype == torch.bfloat16 else p.float().double() for p in s["pools"]]
    for b, base in enumerate(s["base"]):
        at, place = 0, 0
        while at is not None:
            (p, o), (r, u) = divmod(base + place, PAGE), divmod(base + at, PAGE)
            for x in pools:
                if c["layout"] in LOCAL:
                    x[table[b][p], :, :, o] = x[table[b][r], :, :, u].clone()
                else:
                    x[table[b][p], o // 8, :, o % 8] = x[table[b][r], u // 8, :, u % 8].clone()
            at = next((i for i in range(at + 1, n)
                       if parent[b * n + i] == at and draft[b * n + i] == target[b * n + at]), None)
            place += 1
    return [None, None, None, None] + pools


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_append": _exact_norm, "tree_local": _exact_tree, "tree_global": _exact_tree,
            "commit": _exact_commit}[case["op"]](s)
