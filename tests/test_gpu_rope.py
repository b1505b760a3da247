"""gw_rope_rows and gw_rope_cs_scaled against their definitions in float64.

Tolerances.  A rotated value is fl(fl(x0 c) -+ fl(x1 s)) in binary32: three
roundings, so it is off by at most 2^-24 (|x0 c| + |x1 s|) from the products
and 2^-24 of the result from the sum, together below 2^-23 (|x0 c| + |x1 s|)
(1 + 2^-20); the rounding to the element type adds eps/2 of the value, and
half of the smallest subnormal for fp16.  A table entry is one rounding
(2^-24 relative) of an angle in float64 (frequency and product each within an
ulp or two: 2^-51 of the angle) whose cosine and sine are good to 2^-36.
"""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _split(x, rot, interleaved):
    return (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _want(x, pos, cs, rot, interleaved, inverse):
    """(float64 rows, per-element sum of the products' magnitudes)."""
    x = x.double().cpu()
    c, s = cs.double().cpu()[pos.long().cpu()][:, None].unbind(-1)
    if inverse:
        s = -s
    x0, x1 = _split(x, rot, interleaved)
    y, mag = x.clone(), torch.zeros_like(x)
    for t, v0, v1 in ((y, x0 * c - x1 * s, x1 * c + x0 * s), (mag, (x0 * c).abs() + (x1 * s).abs(),
                                                             (x1 * c).abs() + (x0 * s).abs())):
        a, b = _split(t, rot, interleaved)
        a.copy_(v0)
        b.copy_(v1)
    return y, mag


def _check(got, x, pos, cs, rot, interleaved, inverse):
    want, mag = _want(x, pos, cs, rot, interleaved, inverse)
    kind = got.dtype
    first = 2.0 ** -23 * mag * (1 + 2.0 ** -20)
    half_eps = 0.0 if kind == torch.float32 else torch.finfo(kind).eps / 2
    tol = first + half_eps * (want.abs() + first) + (2.0 ** -25 if kind == torch.float16 else 0.0)
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())
    if rot < x.shape[-1]:
        assert torch.equal(got[..., rot:], x[..., rot:])


def _inputs(rows, heads, dim, rot, kind, max_pos, seed=1, theta=1e4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, heads, dim, generator=g, device="cuda").to(DT[kind])
    pos = torch.randint(0, max_pos, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return x, pos, gw.rope_cs_scaled(theta, rot, dim, max_pos)


SHAPES = [  # rows, heads, dim, rot
    (1, 1, 2, 2), (1, 32, 256, 256), (3, 5, 64, 64), (7, 1, 72, 70), (16, 32, 512, 128), (5, 3, 80, 16), (33, 2, 96, 48),
    (2, 31, 1024, 1024), (4, 4, 1024, 6), (129, 8, 128, 32), (17, 2, 9, 6), (300, 7, 40, 24), (1, 3, 512, 510),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_match_definition(shape, kind, interleaved):
    rows, heads, dim, rot = shape
    for inverse in (False, True):
        x, pos, cs = _inputs(rows, heads, dim, rot, kind, 5000) if rot <= 512 else (*_inputs(
            rows, heads, dim, 2, kind, 50)[:2], torch.randn(50, rot // 2, 2, device="cuda"))
        got = gw.rope_rows(x, pos, cs, rot_dim=rot, interleaved=interleaved, inverse=inverse)
        _check(got, x, pos, cs, rot, interleaved, inverse)
        here = x.clone()
        assert gw.rope_rows(here, pos, cs, out=here, rot_dim=rot, interleaved=interleaved, inverse=inverse) is here
        assert torch.equal(here, got)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,pad,shift", [(128, 128, 0, 0), (128, 64, 8, 0), (128, 64, 3, 0), (96, 48, 16, 1),
                                               (64, 64, 0, 5)])
def test_strides_and_alignments(kind, interleaved, dim, rot, pad, shift):
    """Slices of packed projections, shifted bases, head-major and broadcast
    rows; what lies between the rows is left alone."""
    rows, heads = 11, 3
    x0, pos, cs = _inputs(rows, heads, dim, rot, kind, 300)
    want = gw.rope_rows(x0, pos, cs, rot_dim=rot, interleaved=interleaved)

    def room(n, k, gap):
        flat = torch.full((n * (k * (dim + gap) + gap) + shift + 8,), 7.0, dtype=DT[kind], device="cuda")
        v = flat[shift:shift + n * (k * (dim + gap) + gap)].view(n, k * (dim + gap) + gap)
        return flat, v[:, :k * (dim + gap)].view(n, k, dim + gap)[..., :dim]

    fx, x = room(rows, heads, pad)
    x.copy_(x0)
    fy, y = room(rows, heads, pad)
    gw.rope_rows(x, pos, cs, out=y, rot_dim=rot, interleaved=interleaved)
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert bool((fy == 7.0).all())
    fh, hm = room(heads, rows, pad)                      # head-major
    gw.rope_rows(x, pos, cs, out=hm.transpose(0, 1), rot_dim=rot, interleaved=interleaved)
    assert torch.equal(hm.transpose(0, 1), want)
    gw.rope_rows(x, pos, cs, out=x, rot_dim=rot, interleaved=interleaved)
    assert torch.equal(x, want)
    x.fill_(7.0)
    assert bool((fx == 7.0).all())
    one = x0[:1, :1].expand(rows, heads, dim)            # one row for all positions and heads
    got = gw.rope_rows(one, pos, cs, rot_dim=rot, interleaved=interleaved)
    assert torch.equal(got, gw.rope_rows(one.contiguous(), pos, cs, rot_dim=rot, interleaved=interleaved))


def test_half_pairs_are_the_appends_bits():
    """Rows rotated here are the bytes that gw_kv_append stores."""
    for layout, heads, dim, rot, theta in (("local", 4, 256, 256, 1e4), ("full", 1, 512, 128, 1e6)):
        k, pos, _ = _inputs(16, heads, dim, rot, "bf16", 4096)
        cs = gw.rope_cs(theta, rot, dim, 4096)
        pool = gw.KVPool(layout, "bf16", 1, heads)
        slot = G.i32(range(16))
        gw.kv_append(pool, k, k, slot, pos, cs)
        def stored():
            page = pool.data.view(torch.bfloat16)
            if layout == "local":
                return page.view(heads, 2, 16, dim)[:, 0].transpose(0, 1).contiguous()
            return page.view(2, 128, 8, 8).permute(0, 2, 1, 3).reshape(16, 1, 1024)[..., :512].contiguous()

        y = gw.rope_rows(k, pos, cs, rot_dim=rot)
        assert torch.equal(stored().view(torch.int16), y.view(torch.int16))
        # interleaved rows, appended as they are at position 0
        z = gw.rope_rows(k, pos, cs, rot_dim=rot, interleaved=True)
        gw.kv_append(pool, z, k, slot, torch.zeros_like(pos), cs)
        assert torch.equal(stored(), z)


def test_rows_and_tables_beyond_2_31_elements():
    rows, heads, dim = 70001, 64, 512
    assert rows * heads * dim > 2 ** 31
    x = torch.ones(1, heads, dim, dtype=torch.bfloat16, device="cuda").expand(rows, heads, dim)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") % 1000
    cs = gw.rope_cs_scaled(1e6, 128, dim, 1000)
    y = gw.rope_rows(x, pos, cs, rot_dim=128)
    last = slice(rows - 3, rows)
    _check(y[last], x[last], pos[last], cs, 128, False, False)
    del y
    max_pos, half = 9000001, 128
    assert max_pos * half * 2 > 2 ** 31
    got = gw.rope_cs_scaled(1e4, 2 * half, 256, max_pos)[-2:].double().cpu().numpy()
    ang = np.arange(max_pos - 2, max_pos, dtype=np.float64)[:, None] * _freq(1e4, 2 * half, 256, "none", 1, 0, 0, 0)
    want = np.stack([np.cos(ang), np.sin(ang)], -1)
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -51 * ang[..., None] + 2.0 ** -36)


def test_bad_positions_leave_their_rows():
    x, _, cs = _inputs(6, 2, 64, 64, "bf16", 10)
    pos = G.i32([0, -1, 9, 10, 2 ** 31 - 1, 3])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 5.0)
    gw.rope_rows(x, pos, cs, out=y, dev_status=status)
    assert int(status) == gw.GW_DEV_POS_RANGE
    bad = torch.tensor([1, 3, 4], device="cuda")
    assert bool((y[bad] == 5.0).all())
    good = torch.tensor([0, 2, 5], device="cuda")
    _check(y[good], x[good], pos[good], cs, 64, False, False)
    assert int(gw.rope_rows(x[:0], pos[:0], cs).numel()) == 0


def test_special_values_stay_in_their_pair():
    x, pos, cs = _inputs(4, 2, 64, 32, "fp32", 100)
    pos.fill_(7)
    clean = gw.rope_rows(x, pos, cs, rot_dim=32)
    x[1, 0, 3] = float("nan")
    x[2, 1, 40] = float("inf")
    got = gw.rope_rows(x, pos, cs, rot_dim=32)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 0, 3] = touched[1, 0, 19] = touched[2, 1, 40] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert bool(got[1, 0, [3, 19]].isnan().all()) and float(got[2, 1, 40]) == float("inf")


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """d/dx sum(g * rotate(x)) against differences.  The map is linear, so a
    step of one is exact but for rounding: each rotated value is off by at
    most 2^-23 of (|x0 c| + |x1 s|) <= 2^-23 * 16 here, on both sides."""
    rows, heads, dim, rot = 2, 1, 10, 8
    x, pos, cs = _inputs(rows, heads, dim, rot, "fp32", 50)
    g = torch.randn(rows, heads, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    grad = gw.rope_rows(g, pos, cs, rot_dim=rot, interleaved=interleaved, inverse=True)
    _check(grad, g, pos, cs, rot, interleaved, True)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = 1.0
        e = e.view_as(x)
        up = gw.rope_rows(x + e, pos, cs, rot_dim=rot, interleaved=interleaved).double()
        down = gw.rope_rows(x - e, pos, cs, rot_dim=rot, interleaved=interleaved).double()
        step = float((g.double() * (up - down)).sum() / 2)
        # the shifted inputs x +- 1 are rounded too: 2^-22 covers them and the two sides
        assert abs(step - float(grad.view(-1)[i])) <= 2.0 ** -22 * 16 * float(g.abs().sum())


def test_graph_stream_and_launch_settings():
    x, pos, cs = _inputs(40, 8, 128, 64, "bf16", 500)
    want = gw.rope_rows(x, pos, cs, rot_dim=64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    gw.rope_rows(x, pos, cs, out=y, rot_dim=64, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    buf = torch.zeros_like(x)
    tab = torch.zeros(500, 32, 2, device="cuda")
    with torch.cuda.graph(graph):
        gw.rope_cs_scaled(1e4, 64, 128, 500, out=tab)
        gw.rope_rows(buf, pos, tab, out=y, rot_dim=64)
    for _ in range(2):
        y.zero_()
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    try:
        gw.set_early_inputs(True)
        gw.set_max_ctas(3)
        assert torch.equal(gw.rope_rows(x, pos, cs, rot_dim=64), want)
        gw.set_early_launch(False)
        assert torch.equal(gw.rope_rows(x, pos, cs, rot_dim=64), want)
    finally:
        gw.set_early_inputs(False)
        gw.set_max_ctas(0)
        gw.set_early_launch(True)


def _freq(theta, rot, dim, kind, factor, low, high, orig):
    out = []
    for i in range(rot // 2):
        t = theta * factor ** (dim / (dim - 2)) if kind == "ntk" else theta
        f = t ** (-2.0 * i / dim)
        if kind == "linear":
            f = f / factor
        if kind == "ramp":
            keep = min(1.0, max(0.0, (orig * f / (2 * np.pi) - low) / (high - low)))
            f = f * keep + (1 - keep) * f / factor
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("kind,factor,amp", [("none", 1.0, 1.0), ("none", 1.0, 0.5), ("linear", 4.0, 1.0),
                                             ("linear", 0.5, 1.0), ("ntk", 8.0, 1.0), ("ramp", 16.0, 1.2772)])
@pytest.mark.parametrize("theta,rot,dim,max_pos", [(1e4, 256, 256, 3001), (1e6, 128, 512, 150000), (5e5, 2, 64, 1),
                                                   (1e4, 6, 80, 700), (1e4, 512, 512, 129), (1e4, 510, 1024, 64),
                                                   (1e4, 64, 64, 65)])
def test_scaled_table(kind, factor, amp, theta, rot, dim, max_pos):
    low, high, orig = 1.0, 32.0, 8192
    room = torch.full((max_pos * rot + 64,), 3.0, device="cuda")
    got = gw.rope_cs_scaled(theta, rot, dim, max_pos, kind=kind, factor=factor, low=low, high=high, orig_max_pos=orig,
                            amplitude=amp, out=room[:max_pos * rot].view(max_pos, rot // 2, 2))
    assert bool((room[max_pos * rot:] == 3.0).all())
    ang = np.arange(max_pos, dtype=np.float64)[:, None] * _freq(theta, rot, dim, kind, factor, low, high, orig)
    want = amp * np.stack([np.cos(ang), np.sin(ang)], -1)
    tol = 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(want) + amp * (2.0 ** -51 * ang[..., None] + 2.0 ** -36)
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= tol), float(np.max(off - tol))


def test_unscaled_table_is_rope_cs():
    """Both build the unscaled table; they may differ by the last bit where
    the two angles' float64 roundings differ."""
    a, b = gw.rope_cs(1e6, 128, 512, 70000), gw.rope_cs_scaled(1e6, 128, 512, 70000)
    ang = 70000.0
    assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -23 + 2.0 ** -50 * ang


def test_binding_refuses():
    x, pos, cs = _inputs(4, 2, 64, 64, "bf16", 10)
    for call in (lambda: gw.rope_rows(x, pos, None), lambda: gw.rope_rows(x, pos.long(), cs), lambda: gw.rope_rows(x[0], pos, cs),
                 lambda: gw.rope_rows(x, pos[:3], cs), lambda: gw.rope_rows(x, pos, cs, rot_dim=32),
                 lambda: gw.rope_rows(x.double(), pos, cs), lambda: gw.rope_rows(x, pos, cs, out=x.float()),
                 lambda: gw.rope_rows(x[..., ::2], pos, cs[:, :16].contiguous()), lambda: gw.rope_rows(x, pos, cs.cpu()),
                 lambda: gw.rope_rows(x, pos, cs, out=x[:, :1].expand(4, 2, 64)),
                 lambda: gw.rope_rows(x[:3], pos[:3], cs, out=x[1:]), lambda: gw.rope_cs_scaled(1e4, 64, 128, 10, out=cs[:9])):
        with pytest.raises(gw.GwError):
            call()
