"""The rows of gw_decode_attn_global_acc where softmax weights held in few bits
would show: values that a row has to give back, and long tails behind a token
that draws nearly everything.

Tolerances.  The weights enter P.V as sums of terms: on bf16 pools two bf16
terms, the first cut off (less than 2^-7 of a weight is left, 2^-8 of that is
the second one's rounding), good to 2^-15; on e4m3 pools a weight, scaled so
that the largest of a unit is at least 2^7, is rounded to fp16 (2^-11) and cut
into four e5m2 terms, which lose what lies below 2^-16, 2^-23 of the largest.
A row is a sum of such weights times values over their sum in float32; the
tensor cores' sums are off by at most 2^-23 a step of 16 tokens and term, 2^-15
for the units of up to 1024 tokens here.  Then comes the row's rounding to
bf16, 2^-8 of it.
"""

import math

import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

LAYOUTS = ["folded", "full", "folded_e4m3"]
ROW = {"folded": (640, 8, torch.bfloat16), "full": (1024, 8, torch.bfloat16), "folded_e4m3": (640, 16, torch.float8_e4m3fn)}
WEIGHT = {"folded": (2.0 ** -15, 0.0), "full": (2.0 ** -15, 0.0), "folded_e4m3": (2.0 ** -11, 2.0 ** -23)}  # relative, of the largest


def _rows(layout, k_rot, v):
    """Cache rows of keys k_rot [n, 128] and values v [n, 512]; on a full
    pool the keys' other dims are the values', as on the folded ones."""
    return torch.cat([k_rot, v[:, 128:], v], 1) if layout == "full" else torch.cat([v, k_rot], 1)


def _attend(layout, seqs, q, scale, plain=False):
    """Rows [n, heads, 512], lse and weights of q [n, heads, 512] over
    sequences of cache rows."""
    row, blk, kind = ROW[layout]
    need = [(len(x) + 15) // 16 for x in seqs]
    pool = gw.KVPool(layout, "e4m3" if layout == "folded_e4m3" else "bf16", sum(need))
    bt = torch.full((len(seqs), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(seqs):
        p = torch.zeros(need[b] * 16, row, device="cuda")
        p[:len(x)] = x
        p = p.to(torch.bfloat16).to(kind).view(torch.uint8).view(need[b], 2, 8, row // blk, 16).permute(0, 1, 3, 2, 4)
        pool.data.view(-1, 2, row // blk, 8, 16)[at:at + need[b]] = p
        bt[b, :need[b]] = torch.arange(at, at + need[b])
        at += need[b]
    bt, lens = bt.cuda(), G.i32([len(x) for x in seqs])
    out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = G.i32(range(len(seqs) + 1))
    if plain:
        ws = gw.alloc_workspace(pool, q.shape[1], len(seqs), bt.shape[1])
        gw.decode_attn_global(pool, q, out, cu, lens, bt, ws, scale, 1, status)
        assert int(status) == 0
        return out
    acc, lse = torch.zeros(len(seqs), bt.shape[1] * 16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    ws = gw.alloc_workspace_acc(pool, q.shape[1], len(seqs), bt.shape[1])
    gw.decode_attn_global_acc(pool, q, out, lse, acc, cu, lens, bt, ws, 1.0, scale, status)
    assert int(status) == 0
    return out, lse, acc


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("heads", [8, 16, 32])
@pytest.mark.parametrize("spread", [0.1, 1.0, 3.0])
def test_equal_values_come_back(layout, heads, spread):
    """Where every token holds the value 1 a row is exactly 1, flat or peaked:
    the weights that are contracted and those that are summed agree to better
    than 2^-10, and 1 - 2^-10 rounds to 1 (bf16's step below 1 is 2^-8)."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    lens = [2, 3, 17, 65, 300, 900, 5000]
    seqs = [_rows(layout, torch.randn(n, 128, generator=g, device="cuda"), torch.ones(n, 512, device="cuda"))
            for n in lens]
    q = torch.randn(len(lens), heads, 512, generator=g, device="cuda").to(torch.bfloat16)
    out, _, _ = _attend(layout, seqs, q, spread / 11)    # logits of standard deviation `spread`
    assert bool((out == 1).all()), float((out.float() - 1).abs().max())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_later_token_that_dominates(layout):
    """The same for a token of a later tile that is ahead of the first tile's
    maximum by less than makes it the new reference, at weights all over an
    octave: rounded to bf16 alone they are off by up to 2^-8."""
    k = torch.full((65, 128), 0.0, device="cuda")
    k[1:64, 0] = -64.0
    k[64, 0] = 8.0
    rows = _rows(layout, k, torch.ones(65, 512, device="cuda"))
    q = torch.zeros(1, 8, 512, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    for octave in range(8):
        for i in range(16):
            ahead = 2.0 ** octave * (1 + (i + 0.9) * 2.0 ** -10 if i < 8 else 1 + (i - 7.5) / 8.5)
            out, _, _ = _attend(layout, [rows], q, math.log(ahead) / 8)
            assert bool((out == 1).all()), (ahead, float(out[0, 0, 0]))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("nats", [4.0, 8.0, 11.1, 12.0, 13.0, 16.0])
@pytest.mark.parametrize("others", ["near", "far"])
def test_a_tail_behind_one_token(layout, nats, others):
    """131072 tokens, the first one `nats` ahead: of all the others, or of its
    unit's while the rest are far behind.  The tail's own values reach the row."""
    n, unit, heads = 131072, 1024, 8
    k = torch.zeros(n, 128, device="cuda")
    k[0, 0] = 8.0
    if others == "far":
        k[unit:, 0] = -64.0
    q = torch.zeros(1, heads, 512, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = nats / 8
    e = k[:, 0].double() * scale
    w = torch.softmax(e, 0)
    rel, floor = WEIGHT[layout]
    for first, tail in ((1.0, 1.0), (0.0, 1.0), (-1.0, 1.0), (1.0, 0.0)):
        v = torch.full((n, 512), tail, device="cuda")
        v[0] = first
        out, lse, acc = _attend(layout, [_rows(layout, k, v)], q, scale)
        want = float((w * v[:, 0].double()).sum())
        size = float((w * v[:, 0].double().abs()).sum())
        tol = 2.0 ** -8 * abs(want) + (1 + 2.0 ** -8) * ((rel + 2.0 ** -15) * size + unit * floor * float(w.max()) * abs(tail))
        off = float((out.double() - want).abs().max())
        assert off <= tol, (first, tail, want, off, tol)
        assert abs(float(lse[0, 0]) - float(torch.logsumexp(e, 0))) <= 2.0 ** -17 * (1 + nats)
        # below float32's smallest normal number, 2^-126, a weight may be any number up to that
        assert bool(((acc[0].double() - heads * w).abs() <= 2.0 ** -17 * heads * w * (1 + nats) + heads * 2.0 ** -126).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_rows_against_float64(layout, spread):
    """Random rows, element by element.  A logit is off by at most 2^-17 of
    sum |q k| scale (the weights' tests), a weight by twice that and by its
    terms' bound."""
    g = torch.Generator(device="cuda").manual_seed(5)
    lens, heads, scale = [1, 2, 40, 700, 3000], 16, spread / math.sqrt(512)
    kind = ROW[layout][2]
    seqs = [_rows(layout, torch.randn(n, 128, generator=g, device="cuda"), torch.randn(n, 512, generator=g, device="cuda") + 0.5)
            .to(torch.bfloat16).to(kind).float() for n in lens]
    q = torch.randn(len(lens), heads, 512, generator=g, device="cuda").to(torch.bfloat16)
    out, _, _ = _attend(layout, seqs, q, scale)
    rel, floor = WEIGHT[layout]
    for b, x in enumerate(seqs):
        x = x.double()
        k, v = (x[:, :512], x[:, 512:]) if layout == "full" else (torch.cat([x[:, 512:], x[:, 128:512]], 1), x[:, :512])
        e = q[b].double() @ k.T * scale
        w = torch.softmax(e, -1)
        logit = 2.0 ** -16 * float((q[b].double().abs() @ k.T.abs()).max()) * scale + 2.0 ** -22 * float(e.abs().max())
        want, size = w @ v, w @ v.abs()
        tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (
            (rel + logit + 2.0 ** -15) * size + floor * w.amax(-1, keepdim=True) * v.abs().sum(0))
        off = (out[b].double() - want).abs()
        assert bool((off <= tol).all()), (b, float((off - tol).max()))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("at", [0, 70, 699])
def test_a_key_of_nan_stays_with_its_token(layout, at):
    """One token's key holds a NaN: every head's logit of it is NaN, so its
    acc is, the rows are, and the other tokens' weights take nothing."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = _rows(layout, torch.randn(700, 128, generator=g, device="cuda"), torch.randn(700, 512, generator=g, device="cuda"))
    rows[at, 512 if layout != "full" else 0] = float("nan")
    q = torch.randn(1, 8, 512, generator=g, device="cuda").to(torch.bfloat16)
    out, _, acc = _attend(layout, [rows], q, 0.05)
    assert bool(out.isnan().all()) and bool(acc[0, at].isnan())
    rest = torch.arange(acc.shape[1], device="cuda") != at
    assert bool((acc[0, rest] == 0).all())
