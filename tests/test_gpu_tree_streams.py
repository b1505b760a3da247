"""Tree attention on two streams at once, a workspace each."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import Case

pytestmark = pytest.mark.gpu


def call(c, out, ws, stream):
    d, most = c.dev, max(n for _, n in c.plan)
    if c.layout == "local":
        gw.tree_attn_local(c.pool, c.q, out, d["cu"], d["lens"], d["table"], d["mask"], d["pos"], ws, c.window,
                           max_q_rows=most, stream=stream)
    else:
        gw.tree_attn_global(c.pool, c.q, out, d["cu"], d["lens"], d["table"], d["mask"], ws, max_q_rows=most,
                            stream=stream)


def test_two_streams():
    cases = [Case("folded", [(3000 + 100 * b, 4) for b in range(6)], 8, seed=1),
             Case("full", [(900, 7), (2000, 3)], 8, seed=2),
             Case("folded_e4m3", [(2700, 5), (700, 9)], 16, seed=3),
             Case("local", [(1500, 12), (400, 7), (90, 16)], 8, 4, window=1000, seed=4)]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for first, second in ((0, 3), (1, 2), (0, 0), (2, 3)):
        pairs = []
        for s, k in zip(streams, (first, second)):
            s.wait_stream(torch.cuda.current_stream())
            pairs.append((s, k, cases[k].ws.clone(), [torch.full_like(want[k], float("nan")) for _ in range(10)]))
        torch.cuda.synchronize()
        for i in range(10):
            for s, k, ws, outs in pairs:
                call(cases[k], outs[i], ws, s)
        torch.cuda.synchronize()
        for _, k, _, outs in pairs:
            assert all(torch.equal(o, want[k]) for o in outs), (first, second)
