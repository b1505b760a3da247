"""Outputs that the binding allocates come from the memory of the call's stream."""

import pytest
import torch

from paged_hybrid_attention_gb300 import gw

pytestmark = pytest.mark.gpu


def _stream_of(t):
    return [s["stream"] for s in torch.cuda.memory_snapshot()
            if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]


def test_new_outputs_belong_to_the_calls_stream():
    side = torch.cuda.Stream()
    x = torch.randn(4096, 8, 256, device="cuda")
    pos = torch.arange(4096, dtype=torch.int32, device="cuda")
    torch.empty(1 << 26, device="cuda")  # a free block of the current stream that an output would fit into
    torch.cuda.synchronize()
    cs = gw.rope_cs_scaled(1e4, 256, 256, 4096, stream=side)
    plain = gw.rope_cs(1e4, 256, 256, 4096, stream=side)
    y = gw.rope_rows(x, pos, cs, stream=side)
    side.synchronize()
    assert all(_stream_of(t) == [side.cuda_stream] for t in (cs, plain, y))
    assert torch.equal(y, gw.rope_rows(x, pos, cs))
    assert torch.equal(cs, gw.rope_cs_scaled(1e4, 256, 256, 4096))
    here = gw.rope_rows(x, pos, cs)
    assert _stream_of(here) != [side.cuda_stream]
