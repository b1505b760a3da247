"""Operators around the paged global cache, with the cases they are measured at.

Five operators that a decode loop uses together: the rotation of q rows
(`rope_rows`), its (cos, sin) table for scaled contexts (`rope_table`), global
decode attention that adds up each cached token's attention weight
(`attn_acc`), the choice of the tokens to keep by those weights (`select`) and
the move of the kept rows to the front of their sequence's pages (`compact`).

With `own` false, `run` computes them in plain torch operations; with `own`
true it makes the library's calls.
"""

import math
import random

import torch

own = False

PAGE = 16
ELEM = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# layout of the global cache: elements of a token row, elements of a 16-byte
# block, type, and the dims of a row that hold V
LAYOUT = {
    "folded": (640, 8, torch.bfloat16),
    "full": (1024, 8, torch.bfloat16),
    "folded_e4m3": (640, 16, torch.float8_e4m3fn),
}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # q of one decode step: 16 rows of a local layer (latency)
        dict(name="rope_decode", op="rope_rows", rows=16, heads=32, dim=256, rot=256, pairs="half", type="bf16",
             inverse=False, packed=0, inplace=False, max_pos=8192),
        # q of four 2048-token prompts of a global layer, a view of the packed
        # projection, pairs interleaved
        dict(name="rope_prompt", op="rope_rows", rows=8192, heads=32, dim=512, rot=128, pairs="interleaved",
             type="bf16", inverse=False, packed=2, inplace=False, max_pos=131072),
        # the gradient of a rotation, in 32 bits, an odd number of rows
        dict(name="rope_gradient", op="rope_rows", rows=4093, heads=16, dim=256, rot=256, pairs="half", type="fp32",
             inverse=True, packed=0, inplace=False, max_pos=8192),
        # a local layer's table with positions interpolated
        dict(name="table_linear", op="rope_table", max_pos=32768, rot=256, dim=256, theta=1e4, kind="linear",
             factor=4.0, low=0.0, high=0.0, orig=8192, amplitude=1.0),
        # a global layer's table, scaled by a ramp over the turns of a pair
        dict(name="table_ramp", op="rope_table", max_pos=262144, rot=128, dim=512, theta=1e6, kind="ramp",
             factor=8.0, low=1.0, high=32.0, orig=32768, amplitude=1.2079),
        # two short sequences of the full K and V control cache (latency)
        dict(name="acc_small", op="attn_acc", layout="full", heads=8, batch=2, idle=0, min_len=37, max_len=100,
             decay=1.0),
        # the serving step: 16 sequences of 512 to 8192 tokens
        dict(name="acc_serving", op="attn_acc", layout="folded", heads=32, batch=16, idle=0, min_len=512,
             max_len=8192, decay=1.0),
        # long contexts: 8 sequences of 131072 tokens
        dict(name="acc_long", op="attn_acc", layout="folded", heads=32, batch=8, idle=0, min_len=131072,
             max_len=131072, decay=1.0),
        # the serving step's sequences cut to 2048 tokens
        dict(name="select_serving", op="select", batch=16, min_len=512, max_len=8192, budget=2048, sinks=4,
             recent=256),
        # long contexts cut to a quarter
        dict(name="select_long", op="select", batch=8, min_len=131072, max_len=131072, budget=32768, sinks=16,
             recent=1024),
        # the rows that stay on the e4m3 cache, copied out of pages that are shared
        dict(name="compact_copy", op="compact", layout="folded_e4m3", batch=16, min_len=512, max_len=8192, budget=2048,
             copy=True),
        # long contexts cut to a quarter in their own pages
        dict(name="compact_long", op="compact", layout="folded", batch=8, min_len=131072, max_len=131072,
             budget=32768, copy=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_rows", "rope_table", "attn_acc", "attn_acc", "select", "compact"])
    if op == "rope_rows":
        dim = rng.choice([64, 72, 80, 96, 128, 256, 512])
        heads = rng.choice([1, 2, 3, 4, 8, 16, 31, 32])
        kind = rng.choice(["bf16", "fp16", "fp32"])
        rows = _log(rng, 1, max(1, min(16384, (1 << 27) // (heads * dim))))
        return dict(op=op, rows=rows, heads=heads, dim=dim, rot=2 * rng.randint(1, dim // 2),
                    pairs=rng.choice(["half", "interleaved"]), type=kind, inverse=rng.random() < 0.5,
                    packed=rng.choice([0, 0, 1, 2]), inplace=rng.random() < 0.4, max_pos=_log(rng, 1, 32768))
    if op == "rope_table":
        dim = rng.choice([64, 128, 256, 512])
        return dict(op=op, max_pos=_log(rng, 16, 200000), rot=2 * rng.randint(1, min(dim, 256) // 2), dim=dim,
                    theta=rng.choice([1e4, 5e5, 1e6]), kind=rng.choice(["none", "linear", "ntk", "ramp"]),
                    factor=rng.uniform(1.0, 32.0), low=rng.uniform(0.5, 2.0), high=rng.uniform(8.0, 40.0),
                    orig=_log(rng, 2048, 32768), amplitude=rng.uniform(1.0, 1.4))
    batch = _log(rng, 1, 64)
    max_len = _log(rng, 1, min(131072, (1 << 19) // batch))
    min_len = rng.randint(1, max_len)
    if op == "attn_acc":
        return dict(op=op, layout=rng.choice(list(LAYOUT)), heads=rng.choice([8, 16, 32]), batch=batch,
                    idle=rng.randint(0, batch // 2), min_len=min_len, max_len=max_len,
                    decay=rng.choice([0.0, 0.9, 1.0]))
    budget = rng.randint(1, max_len)
    if op == "select":
        max_len = max(64, max_len)
        budget = rng.randint(8, max_len // 2)
        sinks = rng.randint(0, min(64, budget // 4))
        return dict(op=op, batch=batch, min_len=min_len, max_len=max_len, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget // 2))
    return dict(op=op, layout=rng.choice(list(LAYOUT)), batch=batch, min_len=min_len, max_len=max_len,
                budget=budget, copy=rng.random() < 0.4)


# --------------------------------------------------------------- the inputs
def _lens(case):
    """The batch's lengths: spread evenly from min_len to max_len."""
    n = case["batch"] - case.get("idle", 0)
    lo, hi = case["min_len"], case["max_len"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(g, *shape):
    """Accumulated attention weights: a long tail, a third of them with no
    weight at all (ties)."""
    w = torch.exp(torch.randn(*shape, generator=g, device="cuda") * 2 - 6)
    return torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.3, torch.zeros_like(w), w)


def _cache(case, seed, g, copies=1):
    """A pool whose pages the sequences hold in scattered order, their lengths
    and block tables (`copies` of them, over different pages)."""
    lens = _lens(case)
    random.Random(seed).shuffle(lens)
    lens += [0] * (case["batch"] - len(lens))
    row, blk, kind = LAYOUT[case["layout"]]
    need = [(n + PAGE - 1) // PAGE for n in lens]
    width = max(need)
    total = sum(need) * copies
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    ends = [sum(need[:i + 1]) for i in range(len(need))]
    first = torch.tensor([e - n for e, n in zip(ends, need)], device="cuda")[:, None]
    count = torch.tensor(need, device="cuda")[:, None]
    col = torch.arange(width, device="cuda")[None, :]
    tables = []
    for c in range(copies):
        at = (first + col + c * sum(need)).clamp(max=total - 1)
        tables.append(torch.where(col < count, perm[at], torch.full_like(perm[at], -1)).contiguous())
    pool = torch.randn(total, 2, row // blk, 8, blk, generator=g, device="cuda", dtype=torch.bfloat16)
    if kind != torch.bfloat16:
        pool = pool.to(kind)
    return pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), tables, lens


def _handle(case, s):
    """What a program that uses the library keeps for a cache: its pool
    descriptor and the call's workspace."""
    from paged_hybrid_attention_gb300 import gw
    pool = gw.KVPool(case["layout"], "e4m3" if case["layout"] == "folded_e4m3" else "bf16", s["pool"].shape[0],
                     storage=s["pool"].view(torch.uint8).view(-1))
    ws = None
    if case["op"] == "attn_acc":
        ws = gw.alloc_workspace_acc(pool, case["heads"], case["batch"], s["table"].shape[1])
    return pool, ws


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "rope_rows":
        kind = ELEM[case["type"]]
        x = torch.randn(case["rows"], case["heads"] + case["packed"], case["dim"], generator=g, device="cuda").to(kind)
        s["x"] = x[:, :case["heads"]]
        s["out"] = s["x"] if case["inplace"] else torch.empty(case["rows"], case["heads"], case["dim"], dtype=kind,
                                                              device="cuda")
        s["pos"] = torch.randint(0, case["max_pos"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
        f = 1e4 ** (torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) * -2 / case["dim"])
        a = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * f
        s["cs"] = torch.stack([a.cos(), a.sin()], -1).float()
    elif op == "rope_table":
        # no data goes in: the seed moves theta a little, so that tables differ
        s["theta"] = case["theta"] * (1 + random.Random(seed).randrange(1, 1 << 20) * 2.0 ** -22)
        s["out"] = torch.empty(case["max_pos"], case["rot"] // 2, 2, device="cuda")
    elif op == "attn_acc":
        s["pool"], s["lens"], (s["table"],), _ = _cache(case, seed, g)
        rows = case["batch"] - case["idle"]
        s["q"] = torch.randn(rows, case["heads"], 512, generator=g, device="cuda", dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, case["heads"], device="cuda")
        s["acc"] = _weights(g, case["batch"], s["table"].shape[1] * PAGE)
        s["cu"] = torch.arange(case["batch"] + 1, device="cuda", dtype=torch.int32).clamp(max=rows)
        s["handle"] = _handle(case, s) if own else None
    elif op == "select":
        lens = _lens(case)
        random.Random(seed).shuffle(lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["acc"] = _weights(g, case["batch"], case["max_len"])
        s["keep"] = torch.full((case["batch"], case["budget"]), -1, dtype=torch.int32, device="cuda")
        s["keep_lens"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    else:
        s["pool"], s["lens"], tables, lens = _cache(case, seed, g, 2 if case["copy"] else 1)
        s["table"], s["to"] = tables[0], tables[-1]
        s["acc"] = _weights(g, case["batch"], s["table"].shape[1] * PAGE)
        # any subset of the budget's size, ascending, the last token in it
        width = s["acc"].shape[1]
        order = torch.rand(case["batch"], width, generator=g, device="cuda")
        col = torch.arange(width, device="cuda")[None, :]
        order = torch.where(col == s["lens"][:, None] - 1, torch.full_like(order, 2.0), order)
        order = torch.where(col < s["lens"][:, None], order, torch.full_like(order, -1.0))
        top = order.topk(case["budget"], dim=1).indices
        top = torch.where(torch.arange(case["budget"], device="cuda") < s["lens"][:, None], top,
                          torch.full_like(top, width))
        top = top.sort(dim=1).values
        s["keep"] = torch.where(top < width, top, torch.full_like(top, -1)).to(torch.int32)
        s["keep_lens"] = s["lens"].clamp(max=case["budget"]).to(torch.int32)
        s["handle"] = _handle(case, s) if own else None
    return s


# ------------------------------------------------------------------ one pass
def _rope_rows(s):
    c, x, rot = s["case"], s["x"], s["case"]["rot"]
    cs = s["cs"][s["pos"].long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1] * (-1.0 if c["inverse"] else 1.0)
    y = x.float()
    if c["pairs"] == "half":
        x0, x1 = y[..., :rot // 2], y[..., rot // 2:rot]
    else:
        x0, x1 = y[..., :rot:2], y[..., 1:rot:2]
    r0, r1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    r = torch.cat([r0, r1], -1) if c["pairs"] == "half" else torch.stack([r0, r1], -1).flatten(-2)
    if c["inplace"]:
        s["x"][..., :rot] = r.to(x.dtype)
        return s["x"]
    return torch.cat([r.to(x.dtype), x[..., rot:]], -1)


def _rope_table(s):
    c = s["case"]
    theta, factor = s["theta"], c["factor"]
    if c["kind"] == "ntk":
        theta = theta * factor ** (c["dim"] / (c["dim"] - 2))
    f = theta ** (torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * -2 / c["dim"])
    if c["kind"] == "linear":
        f = f / factor
    if c["kind"] == "ramp":
        g = ((f * (c["orig"] / (2 * math.pi)) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = f * (g + (1 - g) / factor)
    a = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * f
    return (torch.stack([a.cos(), a.sin()], -1) * c["amplitude"]).float()


def _rows_of(pool, table):
    """The cached rows that the block tables name, [batch, tokens, row]."""
    r = pool.view(torch.uint8)[table.clamp(min=0).long()].view(pool.dtype)
    return r.permute(0, 1, 2, 4, 3, 5).reshape(table.shape[0], table.shape[1] * PAGE, -1)


def _attn_acc(s):
    c = s["case"]
    n = s["q"].shape[0]
    rows = _rows_of(s["pool"], s["table"][:n]).float()
    if c["layout"] == "full":
        k, v = rows[..., :512], rows[..., 512:]
    else:
        k, v = torch.cat([rows[..., 512:], rows[..., 128:512]], -1), rows[..., :512]
    live = torch.arange(rows.shape[1], device="cuda") < s["lens"][:n, None]
    logit = s["q"].float() @ k.transpose(1, 2) * (1 / math.sqrt(512))
    logit = logit.masked_fill(~live[:, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    w = p / total
    acc = s["acc"][:n]
    old = acc * c["decay"] if c["decay"] else torch.zeros_like(acc)
    acc.copy_(torch.where(live, old + w.sum(1), acc))
    return (w @ v).to(torch.bfloat16), (top + total.log())[..., 0], s["acc"]


def _select(s):
    c, acc = s["case"], s["acc"]
    n, width = acc.shape
    col = torch.arange(width, device="cuda")[None]
    lens = s["lens"][:, None]
    safe = (col < c["sinks"]) | (col >= lens - c["recent"])
    rank = torch.where(safe, 2, 1) * (col < lens)
    value = torch.where(acc.isnan(), torch.full_like(acc, -math.inf), acc)
    order = value.sort(dim=1, descending=True, stable=True).indices
    order = order.gather(1, rank.gather(1, order).sort(dim=1, descending=True, stable=True).indices)
    kept = torch.arange(width, device="cuda")[None] < lens.clamp(max=c["budget"])
    taken = torch.where(kept, order, torch.full_like(order, width)).sort(dim=1).values[:, :c["budget"]]
    s["keep"].copy_(torch.where(taken < width, taken.to(torch.int32), s["keep"]))
    s["keep_lens"].copy_(lens[:, 0].clamp(max=c["budget"]))
    return s["keep"], s["keep_lens"]


def _compact(s):
    keep = s["keep"].long()
    kept = torch.arange(keep.shape[1], device="cuda")[None] < s["keep_lens"][:, None]
    b, i = kept.nonzero(as_tuple=True)
    j = keep[b, i]
    pool = s["pool"].view(torch.uint8)
    src, dst = s["table"][b, j // PAGE].long(), s["to"][b, i // PAGE].long()
    pool[dst, i % PAGE // 8, :, i % 8] = pool[src, j % PAGE // 8, :, j % 8]
    acc, col = s["acc"], torch.arange(s["acc"].shape[1], device="cuda")[None]
    moved = acc[b, j]
    acc.masked_fill_((col >= s["keep_lens"][:, None]) & (col < s["lens"][:, None]), 0.0)
    acc[b, i] = moved
    return s["pool"], acc


def run(s):
    c = s["case"]
    if not own:
        return {"rope_rows": _rope_rows, "rope_table": _rope_table, "attn_acc": _attn_acc, "select": _select,
                "compact": _compact}[c["op"]](s)
    from paged_hybrid_attention_gb300 import gw
    if c["op"] == "rope_rows":
        return gw.rope_rows(s["x"], s["pos"], s["cs"], out=s["out"], rot_dim=c["rot"],
                            interleaved=c["pairs"] == "interleaved", inverse=c["inverse"])
    if c["op"] == "rope_table":
        return gw.rope_cs_scaled(s["theta"], c["rot"], c["dim"], c["max_pos"], kind=c["kind"], factor=c["factor"],
                                 low=c["low"], high=c["high"], orig_max_pos=c["orig"], amplitude=c["amplitude"],
                                 out=s["out"])
    if c["op"] == "attn_acc":
        pool, ws = s["handle"]
        gw.decode_attn_global_acc(pool, s["q"], s["out"], s["lse"], s["acc"], s["cu"], s["lens"], s["table"], ws,
                                  decay=c["decay"])
        return s["out"], s["lse"], s["acc"]
    if c["op"] == "select":
        gw.kv_evict_select(s["acc"], s["lens"], c["budget"], s["keep"], s["keep_lens"], sinks=c["sinks"],
                           recent=c["recent"])
        return s["keep"], s["keep_lens"]
    gw.kv_evict_compact(s["handle"][0], s["table"], s["lens"], s["keep"], s["keep_lens"], acc=s["acc"],
                        dst_block_table=s["to"] if c["copy"] else None)
    return s["pool"], s["acc"]


# ------------------------------------------------------------- what it takes
def work(case):
    op = case["op"]
    if op == "rope_rows":
        size = 4 if case["type"] == "fp32" else 2
        values = case["rows"] * case["heads"]
        moved = values * (case["rot"] if case["inplace"] else case["dim"]) * 2 * size
        table = min(case["rows"], case["max_pos"]) * case["rot"] * 4
        return {"bytes": moved + table + 4 * case["rows"], "flops": values * case["rot"] * 3}
    if op == "rope_table":
        return {"bytes": case["max_pos"] * case["rot"] * 4, "flops": case["max_pos"] * case["rot"] * 2}
    lens = _lens(case)
    if op == "select":
        return {"bytes": 4 * sum(lens) + 4 * sum(min(n, case["budget"]) for n in lens), "flops": sum(lens)}
    row, _, kind = LAYOUT[case["layout"]]
    size = row * torch.empty(0, dtype=kind).element_size()
    if op == "attn_acc":
        heads = len(lens) * case["heads"]
        return {"bytes": sum(lens) * (size + (8 if case["decay"] else 4)) + heads * (2 * 1024 + 4),
                "flops": sum(lens) * case["heads"] * 4 * 512}
    kept = sum(min(n, case["budget"]) for n in lens)
    cut = [n for n in lens if n > case["budget"]]
    moved = kept if case["copy"] else len(cut) * case["budget"]
    return {"bytes": moved * 2 * size + 4 * kept + moved * 8 + 4 * sum(n - case["budget"] for n in cut), "flops": kept}


# ----------------------------------------------- the definitions, in 64 bits
def _exact_rope(s):
    c, rot = s["case"], s["case"]["rot"]
    y = s["x"].double().clone()
    cs = s["cs"].double()[s["pos"].long()]
    turn = torch.complex(cs[..., 0], -cs[..., 1] if c["inverse"] else cs[..., 1])
    even, odd = (slice(0, rot // 2), slice(rot // 2, rot)) if c["pairs"] == "half" else (slice(0, rot, 2),
                                                                                         slice(1, rot, 2))
    for h in range(c["heads"]):
        z = torch.complex(y[:, h, even], y[:, h, odd]) * turn
        y[:, h, even], y[:, h, odd] = z.real, z.imag
    return y


def _exact_table(s):
    c = s["case"]
    freq = []
    for i in range(c["rot"] // 2):
        base = s["theta"] * (c["factor"] ** (c["dim"] / (c["dim"] - 2)) if c["kind"] == "ntk" else 1.0)
        f = base ** (-2.0 * i / c["dim"])
        if c["kind"] == "linear":
            f /= c["factor"]
        elif c["kind"] == "ramp":
            turns = c["orig"] * f / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - c["low"]) / (c["high"] - c["low"])))
            f = f * g + f / c["factor"] * (1 - g)
        freq.append(f)
    f = torch.tensor(freq, dtype=torch.float64)
    out = torch.empty(c["max_pos"], c["rot"] // 2, 2, dtype=torch.float64)
    for p in range(0, c["max_pos"], 8192):
        a = torch.outer(torch.arange(p, min(p + 8192, c["max_pos"]), dtype=torch.float64), f)
        out[p:p + 8192, :, 0], out[p:p + 8192, :, 1] = torch.cos(a) * c["amplitude"], torch.sin(a) * c["amplitude"]
    return out


def _exact_tokens(s, b):
    """The 64-bit rows of sequence b, one token after the other."""
    n = int(s["lens"][b])
    t = torch.arange(n, device="cuda")
    page = s["table"][b].long()[t // PAGE]
    pool = s["pool"] if s["pool"].dtype == torch.bfloat16 else s["pool"].float()
    return pool[page, t % PAGE // 8, :, t % 8].reshape(n, -1).double()


def _exact_attn(s):
    c = s["case"]
    out, lse, acc = [], [], s["acc"].double().clone()
    for b in range(s["q"].shape[0]):
        x = _exact_tokens(s, b)
        v = x[:, 512:] if c["layout"] == "full" else x[:, :512]
        k = x[:, :512].clone()
        if c["layout"] != "full":
            k[:, :128] = x[:, 512:]
        e = s["q"][b].double() @ k.T / math.sqrt(512)
        lse.append(torch.logsumexp(e, -1))
        w = torch.exp(e - lse[-1][:, None])
        out.append(w @ v)
        n = x.shape[0]
        acc[b, :n] = (acc[b, :n] * c["decay"] if c["decay"] else 0.0) + w.sum(0)
        del x, v, k, e, w
    return torch.stack(out), torch.stack(lse), acc


def _exact_compact(s):
    """The move by one step after the other over whole sequences."""
    pool, acc = s["pool"].float(), s["acc"].double().clone()
    was = pool if s["case"]["copy"] else pool.clone()
    for b in range(s["lens"].shape[0]):
        m, n = int(s["keep_lens"][b]), int(s["lens"][b])
        j = s["keep"][b, :m].long()
        i = torch.arange(m, device="cuda")
        p, q = s["table"][b].long()[j // PAGE], s["to"][b].long()[i // PAGE]
        pool[q, i % PAGE // 8, :, i % 8] = was[p, j % PAGE // 8, :, j % 8]
        weights = acc[b, j].clone()
        acc[b, :n] = 0
        acc[b, :m] = weights
    return pool.double(), acc


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return None
    if op == "rope_table":
        return _exact_table(s)
    return {"rope_rows": _exact_rope, "attn_acc": _exact_attn, "compact": _exact_compact}[op](s)
