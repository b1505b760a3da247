"""gw_norm_rope_append against its definition in float64: head layouts, strides,
pool types, rows that are refused."""

import numpy as np
import pytest
import torch

from paged_hybrid_attention_gb300 import gw
from tests.tree_helpers import PAGE, new_pool, to64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def table(rot, dim, theta, max_pos):
    f = theta ** (np.arange(rot // 2) * -2.0 / dim)
    a = np.arange(max_pos)[:, None] * f
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).cuda()


def unit(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)


def turn(x, cs, rot):
    z = (x[..., :rot // 2] + 1j * x[..., rot // 2:rot]) * (cs[..., 0] + 1j * cs[..., 1])[:, None]
    return np.concatenate([z.real, z.imag, x[..., rot:]], -1)


def half_step(x, kind):
    """Half a step of the type at x, and what float32 arithmetic adds: some 30 roundings of 2^-24 of the
    rotated pair, whose elements are at most sqrt(dim) times the weight."""
    if kind == torch.bfloat16:
        return 2.0 ** -8 * np.abs(x) + 2.0 ** -18 * 8
    return np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + 2.0 ** -18 * 8


def make(layout, rows, heads, kv, dtype="bf16", form="packed", seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    dim = 256 if layout == "local" else 512
    size = [heads, kv, kv] if layout == "local" else [heads, 1]
    r = lambda *s: (torch.randn(*s, generator=g) * spread).to(torch.bfloat16).cuda()
    if form == "packed":
        parts = list(r(rows, sum(size), dim).split(size, 1))
    elif form == "apart":
        parts = [r(rows, n, dim) for n in size]
    else:  # head-major, rows with gaps
        parts = [r(n, rows, dim + 8).transpose(0, 1)[..., :dim] for n in size]
    q, k, v = parts[0], parts[1], parts[-1]
    qw, kw = [(1 + 0.3 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
    pages = rows // PAGE + 2
    pool, cells = new_pool(layout, pages, kv, dtype, fill=0x5a)
    slot = torch.randperm(pages * PAGE, generator=g)[:rows].int().cuda()
    pos = torch.randint(0, 500, (rows,), generator=g).int().cuda()
    cs = table(256, 256, 1e4, 500) if layout == "local" else table(128, 512, 1e6, 500)
    return q, k, v, qw, kw, pool, cells, slot, pos, cs


def want_rows(layout, q, k, v, qw, kw, pos, cs, v_norm):
    rot = 256 if layout == "local" else 128
    q, k, v, qw, kw = (to64(x) for x in (q, k, v, qw, kw))
    at = to64(cs)[pos.cpu().numpy()]
    wq, wk = turn(unit(q) * qw, at, rot), turn(unit(k) * kw, at, rot)
    wv = unit(v) if v_norm else v
    if layout in ("folded", "folded_e4m3"):
        wq[..., 128:] *= kw[128:]
    return wq, wk, wv


def check(layout, out, cells, before, slot, wq, wk, wv, rows=None):
    kind = cells.dtype
    rows = np.arange(len(slot)) if rows is None else np.asarray(rows)
    got = to64(out)
    assert np.all(np.abs(got[rows] - wq[rows]) <= half_step(wq[rows], torch.bfloat16))
    s = slot.cpu().numpy()[rows]
    x, touched = to64(cells.view(torch.uint8).view(kind)), np.zeros(tuple(cells.shape), bool)
    if layout == "local":
        gk, gv = x[s // PAGE, :, 0, s % PAGE], x[s // PAGE, :, 1, s % PAGE]
        touched[s // PAGE, :, :, s % PAGE] = True
        parts = ((gk, wk[rows]), (gv, wv[rows]))
    else:
        row = x[s // PAGE, s % PAGE // 8, :, s % PAGE % 8].reshape(len(s), -1)
        touched[s // PAGE, s % PAGE // 8, :, s % PAGE % 8] = True
        k1, v1 = wk[rows][:, 0], wv[rows][:, 0]
        parts = ((row, np.concatenate([k1, v1] if layout == "full" else [v1, k1[:, :128]], 1)),)
    for got, want in parts:
        if kind != torch.bfloat16:
            want = np.clip(want, -448, 448)
        assert np.all(np.abs(got - want) <= half_step(want, kind))
    # nothing else is written
    same = (cells.view(torch.uint8) == before.view(torch.uint8)).cpu().numpy().reshape(tuple(cells.shape) + (-1,)).all(-1)
    assert same[~touched].all()


CASES = [("local", 8, 4, "bf16"), ("local", 32, 16, "e4m3"), ("local", 3, 1, "bf16"), ("local", 5, 5, "e4m3"),
         ("folded", 8, 1, ""), ("full", 16, 1, ""), ("folded_e4m3", 32, 1, "")]


@pytest.mark.parametrize("layout,heads,kv,dtype", CASES)
@pytest.mark.parametrize("rows", [1, 3, 67])
@pytest.mark.parametrize("form", ["packed", "apart", "gaps"])
def test_matches(layout, heads, kv, dtype, rows, form):
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make(layout, rows, heads, kv, dtype or "bf16", form, seed=rows)
    out = torch.full((rows, heads, q.shape[2]), float("nan"), dtype=torch.bfloat16, device="cuda")
    before, status = cells.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS, dev_status=status)
    assert int(status.item()) == 0
    check(layout, out, cells, before, slot, *want_rows(layout, q, k, v, qw, kw, pos, cs, True))


@pytest.mark.parametrize("layout,dtype", [("local", "bf16"), ("local", "e4m3"), ("full", "")])
def test_v_as_it_is(layout, dtype):
    """v_norm 0, on the full layout with v a tensor of its own; values beyond e4m3's range saturate."""
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make(layout, 40, 8, 1, dtype or "bf16", "apart", seed=3, spread=200.0)
    if layout == "full":
        v = torch.randn(40, 1, 512).to(torch.bfloat16).cuda()
    out, before = torch.empty_like(q), cells.clone()
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS, v_norm=False)
    check(layout, out, cells, before, slot, *want_rows(layout, q, k, v, qw, kw, pos, cs, False))


def test_full_pool_with_its_own_v():
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make("full", 21, 8, 1, form="apart", seed=4)
    v = torch.randn(21, 1, 512).to(torch.bfloat16).cuda()
    out, before = torch.empty_like(q), cells.clone()
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS)
    check("full", out, cells, before, slot, *want_rows("full", q, k, v, qw, kw, pos, cs, True))


def test_rows_of_zeros_and_small_values():
    """A head of zeros stays zeros; one far below eps is scaled by 1 / sqrt(eps)."""
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make("local", 8, 8, 2, form="apart", seed=6)
    q[1], k[2], v[3] = 0, 0, 0
    q[4] *= 2.0 ** -20
    out, before = torch.empty_like(q), cells.clone()
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS)
    check("local", out, cells, before, slot, *want_rows("local", q, k, v, qw, kw, pos, cs, True))
    assert (out[1] == 0).all()


@pytest.mark.parametrize("layout", ["local", "folded"])
def test_in_place(layout):
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make(layout, 300, 32, 1, form="apart", seed=7)
    before = cells.clone()
    want = want_rows(layout, q, k, v, qw, kw, pos, cs, True)
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, q, eps=EPS)
    check(layout, q, cells, before, slot, *want)


@pytest.mark.parametrize("layout", ["local", "folded", "full", "folded_e4m3"])
@pytest.mark.parametrize("rows", [9, 200])
def test_rows_out_of_range(layout, rows):
    """A bad slot keeps the row out of the pool, a bad position the whole row."""
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make(layout, rows, 8, 2 if layout == "local" else 1, form="apart", seed=8)
    slot[2], slot[5] = -1, pool.num_pages * PAGE
    before, status = cells.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS, dev_status=status)
    assert int(status.item()) == gw.GW_DEV_SLOT_RANGE
    want = want_rows(layout, q, k, v, qw, kw, pos, cs, True)
    good = [r for r in range(rows) if r not in (2, 5)]
    check(layout, out, cells, before, slot, *want, rows=good)
    assert np.all(np.abs(to64(out) - want[0]) <= half_step(want[0], torch.bfloat16))
    cells.view(torch.uint8).copy_(before.view(torch.uint8))
    safe = pos.clone()
    pos[2], pos[7] = -1, 500
    status.zero_()
    out.fill_(7.0)
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS, dev_status=status)
    assert int(status.item()) == gw.GW_DEV_SLOT_RANGE | gw.GW_DEV_POS_RANGE
    check(layout, out, cells, before, slot, *want, rows=[r for r in good if r != 7])
    assert (out[2] == 7).all() and (out[7] == 7).all() and safe.shape == pos.shape


def test_many_rows_and_early_inputs():
    """Rows whose heads a warp walks in a run, with index inputs read early, captured and replayed."""
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make("local", 2500, 32, 16, "e4m3", seed=9)
    out, before = torch.empty(2500, 32, 256, dtype=torch.bfloat16, device="cuda"), cells.clone()
    want = want_rows("local", q, k, v, qw, kw, pos, cs, True)
    gw.set_early_inputs(True)
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS)
            gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS)
        g.replay()
    finally:
        gw.set_early_inputs(False)
    check("local", out, cells, before, slot, *want)


def test_slots_behind_4_gib():
    q, k, v, qw, kw, _, _, _, pos, cs = make("local", 5, 32, 16, form="apart", seed=10)
    pages = (1 << 32) // 262144 + 4
    pool = gw.KVPool("local", "bf16", pages, 16)
    cells = pool.data.view(torch.bfloat16).view(pages, 16, 2, PAGE, 256)
    slot = torch.tensor([pages * PAGE - 1 - 3 * i for i in range(5)], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    gw.norm_rope_append(pool, q, k, v, qw, kw, slot, pos, cs, out, eps=EPS)
    _, wk, wv = want_rows("local", q, k, v, qw, kw, pos, cs, True)
    s = slot.long()
    gk, gv = to64(cells[s // PAGE, :, 0, s % PAGE]), to64(cells[s // PAGE, :, 1, s % PAGE])
    assert np.all(np.abs(gk - wk) <= half_step(wk, torch.bfloat16))
    assert np.all(np.abs(gv - wv) <= half_step(wv, torch.bfloat16))


def test_binding_refuses():
    q, k, v, qw, kw, pool, cells, slot, pos, cs = make("local", 4, 8, 2, form="apart", seed=1)
    out = torch.empty_like(q)
    args = [pool, q, k, v, qw, kw, slot, pos, cs, out]
    for at, bad in ((1, q.float()), (1, q[:3]), (2, k[:, :1]), (3, v.transpose(1, 2)), (4, qw.bfloat16()), (5, kw[:128]),
                    (6, slot.long()), (7, pos[:3]), (8, cs[:, :64]), (9, out[:, :4]), (9, k), (1, q.cpu())):
        call = list(args)
        call[at] = bad
        with pytest.raises(gw.GwError):
            gw.norm_rope_append(*call)
    with pytest.raises(gw.GwError, match="multiple of 8"):
        odd = torch.zeros(4, 8, 257, dtype=torch.bfloat16, device="cuda")[..., :256]
        gw.norm_rope_append(pool, odd, *args[2:])
    f = make("folded", 4, 8, 1, form="apart", seed=2)
    with pytest.raises(gw.GwError, match="one projection"):
        gw.norm_rope_append(f[5], f[0], f[1], f[1].clone(), f[3], f[4], f[7], f[8], f[9], torch.empty_like(f[0]))


def test_row_layout_is_the_append_s():
    """A unit K row through unit weights: the pool holds what gw_kv_append writes for the normed rows."""
    for layout, kv in (("local", 2), ("folded", 1), ("full", 1)):
        q, k, v, qw, kw, pool, cells, slot, pos, cs = make(layout, 33, 8, kv, form="apart", seed=11)
        dim = q.shape[2]
        sign = torch.where(torch.rand(33, kv, dim, device="cuda") < 0.5, -1.0, 1.0).to(torch.bfloat16)
        one = torch.ones(dim, device="cuda")
        out = torch.empty_like(q)
        # rows of +-1 have mean square 1: with eps below half a unit in the last place they pass as they are
        gw.norm_rope_append(pool, q, sign, sign, one, one, slot, pos, cs, out, eps=1e-12)
        other, want = new_pool(layout, pool.num_pages, kv, fill=0x5a)
        gw.kv_append(other, sign.contiguous(), sign.contiguous(), slot, pos, cs)
        d = (to64(cells) - to64(want))
        # the append's rotation rounds twice more: now and then a neighbour, 2^-7 of values below 2
        assert np.nanmax(np.abs(d)) <= 2.0 ** -7 and (np.abs(d) > 0).mean() < 0.01
        assert (torch.isnan(cells.float()) == torch.isnan(want.float())).all()
