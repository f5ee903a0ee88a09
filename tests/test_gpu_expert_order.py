"""dispatch, combine and combine_grad against their definitions in 64 bits.

Bars, from the arithmetic: a dispatched bf16 row is a copy; its e4m3 codes are half a step
off, 2^-4 of the value or 2^-10 of the scale, and the scale one rounding, 2^-24 (bf16 inputs
are exact).  combine: k fused multiply-adds and one addition in fp32, each off by at
most 2^-24 of a partial sum (at most the sum S of the terms' magnitudes), then half a bf16
step: (k + 1) 2^-24 S + 2^-8 |y|.  d_rows: one rounding to fp32 and one to bf16.  d_w: at most
32 additions in a lane, 8 in the wave and 4 waves, d <= 8192: 50 * 2^-24 S."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain
from routings import device_routing, selections, values

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def wide(t):
    return t.float().cpu().numpy().astype(np.float64)


def rows_of(rng, n, d):
    return torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(bf16)


SHAPES = [(1, 1, 1, 64), (70, 12, 7, 128), (9, 12, 7, 704), (1, 256, 8, 2048), (2, 5, 3, 192), (7, 9, 8, 448), (33, 256, 8, 576),
          (5, 16, 2, 2112), (3, 4, 4, 8192), (129, 3, 1, 1024), (300, 40, 5, 320), (40, 8, 6, 4160)]


def setup(dev, T, E, k, d, room=0):
    rng = np.random.default_rng(T * 131 + E * 7 + d)
    idx, w = selections(rng, T, E, k)
    r, o = device_routing(idx, w, E, dev, room)
    return rng, r, o["inv_perm"].reshape(T, k), w


@pytest.mark.parametrize("T,E,k,d", SHAPES)
def test_dispatch(dev, T, E, k, d):
    rng, r, inv, _ = setup(dev, T, E, k, d, room=T % 2)
    x = rows_of(rng, T, d)
    if T > 2:
        x[1] = 0
        x[2, :64] = 0
    token = np.empty(T * k, np.int64)
    token[inv.reshape(-1)] = np.arange(T * k) // k
    rows, none = q4.dispatch(x.to(dev), r)
    assert none is None and torch.equal(rows.cpu(), x[token])
    room = torch.full((T * k + 1, d), 3.0, device=dev).to(torch.float8_e4m3fn)
    codes, scale = q4.dispatch(x.to(dev), r, rows=room, e4m3=True)
    assert codes is room and bool((room[T * k:].float() == 3.0).all())
    h = wide(x)[token]
    s = plain.group_scales(h)
    assert (np.abs(wide(scale) - s) <= s * 2.0 ** -24).all()
    sc = plain.expand(wide(scale), 1, T * k, d)
    bar = np.maximum(np.abs(h) * 2.0 ** -4, sc * 2.0 ** -10) + np.abs(h) * 2.0 ** -20
    assert (np.abs(values(room[:T * k]) * sc - h) <= bar).all()


@pytest.mark.parametrize("T,E,k,d", SHAPES)
def test_combine(dev, T, E, k, d):
    rng, r, inv, w = setup(dev, T, E, k, d, room=T % 2)
    rows, base = rows_of(rng, T * k, d), rows_of(rng, T, d)
    size = plain.combine(np.abs(wide(rows)), inv, np.abs(w), np.abs(wide(base)))
    for weighted in (True, False):
        for b in (None, base):
            y = q4.combine(rows.to(dev), r, weighted=weighted, base=None if b is None else b.to(dev))
            want = plain.combine(wide(rows), inv, w if weighted else None, None if b is None else wide(b))
            S = size if weighted else plain.combine(np.abs(wide(rows)), inv, None, np.abs(wide(base)))
            bar = (k + 1) * 2.0 ** -24 * S + np.abs(want) * 2.0 ** -8
            assert (np.abs(wide(y) - want) <= bar).all()
    # into base
    bd = base.to(dev)
    assert torch.equal(q4.combine(rows.to(dev), r, base=bd, y=bd), q4.combine(rows.to(dev), r, base=base.to(dev)))


@pytest.mark.parametrize("T,E,k,d", SHAPES)
def test_combine_grad(dev, T, E, k, d):
    rng, r, inv, w = setup(dev, T, E, k, d, room=T % 2)
    rows, dy = rows_of(rng, T * k, d), rows_of(rng, T, d)
    want_rows, want_w = plain.combine_grad(wide(dy), wide(rows), inv, w)
    _, S = plain.combine_grad(np.abs(wide(dy)), np.abs(wide(rows)), inv, w)
    rd = rows.to(dev)
    d_rows, d_w = q4.combine_grad(dy.to(dev), rd, r)
    assert torch.equal(rd.cpu(), rows) and d_w.shape == (T, k)
    assert (np.abs(wide(d_rows) - want_rows) <= np.abs(want_rows) * (2.0 ** -8 + 2.0 ** -23)).all()
    assert (np.abs(wide(d_w) - want_w) <= 50 * 2.0 ** -24 * S).all()
    # in place of the rows
    a, b = q4.combine_grad(dy.to(dev), rd, r, d_rows=rd)
    assert a is rd and torch.equal(a, d_rows) and torch.equal(b, d_w)


def test_gradients_against_differences(dev):
    # L = <combine(rows, w), v> is linear in rows and in w: a step along any direction
    # changes it by the gradient times the step, up to the roundings of y (2^-8 of each)
    T, E, k, d = 6, 5, 3, 192
    rng, r, inv, w = setup(dev, T, E, k, d)
    rows, v = rows_of(rng, T * k, d), rows_of(rng, T, d)
    loss = lambda rr, ww: (plain.combine(rr, inv, ww) * wide(v)).sum()               # noqa: E731
    d_rows, d_w = q4.combine_grad(v.to(dev), rows.to(dev), r)
    u, z = rng.standard_normal((T * k, d)), rng.standard_normal((T, k))
    w64, h = w.astype(np.float64), 2.0 ** -10
    by = (loss(wide(rows) + h * u, w64) - loss(wide(rows) - h * u, w64)) / (2 * h)
    terms = wide(d_rows) * u
    assert abs(terms.sum() - by) <= np.abs(terms).sum() * 2.0 ** -8 + 1e-6
    by = (loss(wide(rows), w64 + h * z) - loss(wide(rows), w64 - h * z)) / (2 * h)
    assert abs((wide(d_w) * z).sum() - by) <= 1e-4 * np.abs(wide(d_w) * z).sum()
    # dispatch: <dispatch(x), g> = <x, combine(g, unweighted)>
    x, g = rows_of(rng, T, d), rows_of(rng, T * k, d)
    there = wide(q4.dispatch(x.to(dev), r)[0]) * wide(g)
    back = wide(x) * wide(q4.combine(g.to(dev), r, weighted=False))
    assert abs(there.sum() - back.sum()) <= np.abs(back).sum() * 2.0 ** -8


def test_weights_of_zero_and_non_finite_rows(dev):
    T, E, k, d = 5, 8, 4, 128
    rng, r, inv, w = setup(dev, T, E, k, d)
    rows = rows_of(rng, T * k, d)
    w[0, 1] = 0.0
    rows[int(inv[0, 1])] = float("nan")      # left out
    w[1, 0] = 0.0
    rows[int(inv[1, 0])] = float("inf")      # left out
    w[2] = 0.0                               # a token without any weight
    rows[int(inv[3, 2]), 5] = float("inf")
    rows[int(inv[4, 0]), 7] = float("nan")
    r.topk_w.copy_(torch.from_numpy(w))
    y = q4.combine(rows.to(dev), r).float().cpu()
    assert y[:2].isfinite().all() and (y[2] == 0).all()
    assert y[3, 5] == float("inf") and y[3, :5].isfinite().all()
    assert y[4, 7].isnan() and y[4, :7].isfinite().all() and y[4, 8:].isfinite().all()
    x = rows_of(rng, T, d)
    x[0, 3], x[1, 4] = float("nan"), float("inf")
    codes, scale = q4.dispatch(x.to(dev), r, e4m3=True)
    at = torch.from_numpy(inv)[:, 0].to(dev)
    c, s = codes.float()[at].cpu(), scale[at].cpu()
    assert c[0].isnan().all() and s[0].isnan().all()
    assert s[1, 0] == float("inf") and c[1, 4].isnan() and (c[1, :4] == 0).all()


def test_indices_out_of_range_stay_in_bounds(dev):
    T, E, k, d = 4, 8, 2, 128
    rng, r, inv, _ = setup(dev, T, E, k, d)
    r.inv_perm.view(-1)[:3] = torch.tensor([-5, 1 << 30, T * k], dtype=torch.int32)
    rows, x = rows_of(rng, T * k, d).to(dev), rows_of(rng, T, d).to(dev)
    y = q4.combine(rows, r, weighted=False)
    want = (rows[0].float() + rows[T * k - 1].float()).to(bf16)
    assert torch.equal(y[0], want)
    guard = torch.zeros(3 * T * k, d, dtype=bf16, device=dev)
    q4.dispatch(x, r, rows=guard[T * k:2 * T * k])
    q4.combine_grad(x, rows, r, d_rows=guard[T * k:2 * T * k])
    torch.cuda.synchronize()
    assert not guard[:T * k].any() and not guard[2 * T * k:].any()


def test_rows_past_32_bits(dev):
    # 2^31 elements of expert rows, 2^32 bytes; tokens in reverse order
    T, E, k, d = 32768, 8, 8, 8192
    idx = np.tile(np.arange(8, dtype=np.int32), (T, 1))
    w = np.random.default_rng(1).random((T, k)).astype(np.float32)
    r, _ = device_routing(idx, w, E, dev)
    inv = torch.arange(T * k - 1, -1, -1, dtype=torch.int32).view(T, k)
    r.inv_perm.view(-1)[:T * k] = inv.view(-1).to(dev)
    x = torch.randn(T, d, device=dev).to(bf16)
    rows, _ = q4.dispatch(x, r)
    codes, scale = q4.dispatch(x, r, e4m3=True)
    y = q4.combine(rows, r)
    at = [0, 1, T // 2, T - 2, T - 1]
    for t in at:
        mine = inv[t].tolist()
        assert all(torch.equal(rows[i], x[t]) for i in mine), t
        h = wide(x[t])
        for i in mine:
            sc = plain.expand(wide(scale[i:i + 1]), 1, 1, d)[0]
            bar = np.maximum(np.abs(h) * 2.0 ** -4, sc * 2.0 ** -10) + np.abs(h) * 2.0 ** -20
            assert (np.abs(values(codes[i:i + 1])[0] * sc - h) <= bar).all(), (t, i)
        want = h * w[t].astype(np.float64).sum()
        size = np.abs(h) * w[t].astype(np.float64).sum()
        assert (np.abs(wide(y[t]) - want) <= (k + 1) * 2.0 ** -24 * size + np.abs(want) * 2.0 ** -8).all()
    _, d_w = q4.combine_grad(x, rows, r, d_rows=rows)
    for t in at:
        h = wide(x[t])
        for s, i in enumerate(inv[t].tolist()):
            want = w[t, s].astype(np.float64) * h
            assert (np.abs(wide(rows[i]) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23)).all()
        assert (np.abs(wide(d_w[t]) - (h * h).sum()) <= 50 * 2.0 ** -24 * (h * h).sum()).all()


def test_streams_and_graphs(dev):
    T, E, k, d = 20, 16, 4, 512
    rng, r, _, _ = setup(dev, T, E, k, d)
    x, rows = rows_of(rng, T, d).to(dev), rows_of(rng, T * k, d).to(dev)
    calls = [lambda **kw: q4.dispatch(x, r, **kw)[0], lambda **kw: q4.combine(rows, r, base=x, **kw),
             lambda **kw: torch.cat([t.float().view(-1) for t in q4.combine_grad(x, rows, r, **kw)])]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c, ref in zip(calls[:2], want):
        got = c(stream=side)
        side.synchronize()
        assert torch.equal(got, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [c() for c in calls]
    for i in range(3):
        x.mul_(-2.0)
        rows.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        for c, got in zip(calls, outs):
            assert torch.equal(c(), got), i
