"""What the binding of the calls around the decode step refuses before the
library sees it: a missing tensor, by name (no GPU needed)."""

import inspect

import pytest
import torch

gw = pytest.importorskip("paged_hybrid_attention_gb300.gw", reason="libgw.so not built")


class Pool:  # of a KVPool what the binding looks at before the call
    data = torch.zeros(16, dtype=torch.uint8)
    desc = None


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _calls():
    return {
        gw.rope_rows: dict(x=torch.zeros(2, 1, 8), pos=_i32(2), rope_cs=torch.zeros(4, 4, 2)),
        gw.decode_attn_global_acc: dict(
            pool=Pool, q=torch.zeros(1, 8, 512, dtype=torch.bfloat16), out=torch.zeros(1, 8, 512, dtype=torch.bfloat16),
            lse=None, acc=torch.zeros(1, 16), cu_q_rows=_i32(2), seq_lens=_i32(1), block_table=_i32(1, 1),
            workspace=torch.zeros(16, dtype=torch.uint8)),
        gw.kv_evict_select: dict(acc=torch.zeros(1, 16), seq_lens=_i32(1), budget=2, keep_idx=_i32(1, 2), keep_lens=_i32(1)),
        gw.kv_evict_compact: dict(pool=Pool, block_table=_i32(1, 1), seq_lens=_i32(1), keep_idx=_i32(1, 2),
                                  keep_lens=_i32(1)),
    }


CASES = [(call, name) for call, args in _calls().items() for name, v in args.items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("call,name", CASES, ids=["%s-%s" % (c.__name__, n) for c, n in CASES])
def test_missing_tensors(call, name):
    args = _calls()[call]
    assert inspect.signature(call).parameters[name].default is inspect.Parameter.empty
    with pytest.raises(gw.GwError, match="not on a CUDA device"):
        call(**args)
    args[name] = None
    with pytest.raises(gw.GwError, match="gw_%s: %s is None" % (call.__name__, name)):
        call(**args)


def test_missing_x_with_an_output():
    with pytest.raises(gw.GwError, match="x is None"):
        gw.rope_rows(None, _i32(2), torch.zeros(4, 4, 2), out=torch.zeros(2, 1, 8))
