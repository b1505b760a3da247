"""Drafted trees on e4m3 pools over a token that draws almost all weight and has no
value of its own (an attention sink): the output is the tail's."""

import math

import numpy as np
import pytest
import torch

from tests.tree_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["local", "folded_e4m3"])
@pytest.mark.parametrize("n", [2, 4, 8, 24])  # few rows and many
@pytest.mark.parametrize("octaves", [11.4, 15.7, 18.3, 20.6, 21.8])
@pytest.mark.parametrize("sink", [3, 100, 700])
def test_sink(layout, n, octaves, sink):
    """Each other token's weight is 2^-octaves of the sink's."""
    local = layout == "local"
    L = 1500
    c = Case(layout, [(L, n)], 8, 1, "e4m3", window=L if local else 0, seed=4)
    first = c.cells.float()
    x = first.clone()
    page, off = int(c.table[0, sink // 16]), sink % 16
    g = torch.Generator().manual_seed(1)
    value = (1 + 0.2 * torch.randn(x.shape, generator=g)).cuda()
    if local:
        x[:, :, 0], x[:, :, 1] = 0, value[:, :, 1]
        x[page, :, 1, off] = 0
        x[page, :, 0, off, 7] = 2.0
    else:
        x[:, :, 32:], x[:, :, :32] = 0, value[:, :, :32]
        x[page, off // 8, :, off % 8] = 0
        x[page, off // 8, 32, off % 8, 7] = 2.0
    x = torch.where(torch.isnan(first), first, x).to(c.cells.dtype)
    c.cells.view(torch.uint8).copy_(x.view(torch.uint8))
    c.q.zero_()
    c.q[:, :, 7] = octaves * math.log(2) / (2 * c.scale)
    c.run()
    # weights down to 2^-22 of the largest hold at least 5 bits and are rounded: within 2^-7 and
    # the roundings that Case.check counts (2^-7 of sum p |v| and 2^-8 of the output)
    want, _ = c.want(0)
    assert float(np.abs(want).min()) > 0
    c.check()
