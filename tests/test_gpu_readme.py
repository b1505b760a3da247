"""The README's verification step runs as it is printed there, and its attention is right."""

import os

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import PAGE, attend, depths, kv_rows, new_pool, seen_by_tree, to64, tree_of, words

pytestmark = pytest.mark.gpu


def block():
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "README.md")) as f:
        text = f.read()
    return text[text.index("Verification of drafted tokens"):].split("```python\n")[1].split("```")[0]


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def test_verification_step():
    rng, g = np.random.default_rng(5), torch.Generator(device="cuda").manual_seed(5)
    heads, kv, plan, width = 32, 16, [(3000, 16), (40, 7)], 200
    B, rows = len(plan), sum(n for _, n in plan)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    weight = lambda n: 1 + 0.1 * torch.randn(n, generator=g, device="cuda")
    trees = [tree_of(rng, n) for _, n in plan]
    cu = np.concatenate([[0], np.cumsum([n for _, n in plan])])
    lens = [L for L, _ in plan]
    pos = np.concatenate([L - n + np.array(depths(t)) for (L, n), t in zip(plan, trees)])
    ns = dict(gw=gw, torch=torch, B=B, P=width, cu_q_rows=i32(cu), seq_lens=i32(lens), pos=i32(pos),
              tree_mask=torch.tensor([w for t in trees for w in words(seen_by_tree(t))], dtype=torch.int64, device="cuda"),
              parent=i32([p for t in trees for p in t]), draft=i32(rng.integers(0, 3, rows)),
              target=i32(rng.integers(0, 3, rows)), path=i32(np.zeros((B, 16))))
    for name in ("path_lens", "next_tokens", "new_lens"):
        ns[name] = i32(np.zeros(B))
    kinds = {"": ("local", kv, 256, 256, 1e4), "g": ("folded", 1, 512, 128, 1e6)}
    cells, tables = {}, {}
    for p, (layout, kvh, dim, rot, theta) in kinds.items():
        pages = B * width
        ns[p + "pool"], cells[p] = new_pool(layout, pages, kvh)
        cells[p].copy_(r(*cells[p].shape))
        tables[p] = rng.permutation(pages).reshape(B, width)
        ns[p + "block_table"] = i32(tables[p])
        x = r(rows, heads + (2 if p == "" else 1) * kvh, dim)
        ns[p + "q"], ns[p + "k"], ns[p + "v"] = x[:, :heads], x[:, heads:heads + kvh], x[:, -kvh:]
        ns[p + "q_norm"], ns[p + "k_norm"] = weight(dim), weight(dim)
        at = [(b, L - n + i) for b, (L, n) in enumerate(plan) for i in range(n)]
        ns[p + "slot"] = i32([tables[p][b, t // PAGE] * PAGE + t % PAGE for b, t in at])
        ns[p + "rope"] = gw.rope_cs(theta, rot, dim, 4096)
        ns[p + "q_rows"] = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda")
        ns[p + "out"] = torch.zeros_like(ns[p + "q_rows"])
    code = block()
    cut = code.index("gw.tree_accept")
    exec(code[:cut], ns)
    for p, (layout, kvh, dim, _, _) in kinds.items():  # before the rows move
        for b, (L, n) in enumerate(plan):
            base, mine = L - n, pos[cu[b]:cu[b + 1]]
            lo = max(0, base - 1023) if p == "" else 0
            at = np.concatenate([np.arange(lo, base), mine])
            sees = np.concatenate([np.ones((n, base - lo), bool), seen_by_tree(trees[b])], 1)
            if p == "":
                sees &= at[None] > mine[:, None] - 1024
            k, v = kv_rows(cells[p], layout, tables[p][b], np.arange(lo, L))
            q = to64(ns[p + "q_rows"][cu[b]:cu[b + 1]])
            want, size = attend(q, k, v, sees, 1 / np.sqrt(dim))
            got = to64(ns[p + "out"][cu[b]:cu[b + 1]])
            # the weights' rounding in numerator and denominator, and the output's: 2^-8 each
            assert (np.abs(got - want) <= 2.0 ** -8 * (2 * size + np.abs(want)) * 1.05 + 1e-6).all()
            assert np.abs(got).max(-1).min() > 0
    exec(code[cut:], ns)
    assert int(ns["status"].item()) == 0
    m = ns["path_lens"].tolist()
    assert all(1 <= x <= n for x, (_, n) in zip(m, plan)) and ns["new_lens"].tolist() == [L - n + x for x, (L, n) in zip(m, plan)]
