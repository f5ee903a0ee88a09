"""moe_add_norm against the formula in 64 bits.

Bars, from the arithmetic:
  - residual_out: one rounding of an exact-enough sum.  fp32: x + residual is one
    fp32 addition, so bit-exact against the same addition on the host; bf16: the
    fp32 sum rounded once, bit-exact too.
  - y: one rounding to bf16 (at most half a step: 2^-8 relative) of an fp32 value
    whose relative error is below 2^-17 (the sum of squares adds at most 32 terms
    per lane and 8 partial sums in sequence, so 40 * 2^-24 and half of that in the
    root, plus six roundings of 2^-24).
  - y8: half an e4m3 step, 2^-4 relative, or half the subnormal step 2^-9 in units
    of the scale; the fp32 value's error (2^-17 relative) moves a value across a
    rounding border by no more than itself.
  - y8_scale: 2^-17 relative like y.
"""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -17
SHAPES = [(1, 64), (1, 2048), (3, 128), (5, 448), (130, 512), (2, 576), (7, 2048), (33, 2112),
          (4, 4096), (3, 4160), (2, 8192), (1500, 1024)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def inputs(T, d, residual, seed=0, plus_one=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    w = ((0.0 if plus_one else 1.0) + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16)
    r = None
    if residual is not None:
        r = (5.0 * torch.randn(T, d, generator=g)).to(residual)
    return x, w, r


def plain(x, w, r, plus_one):
    """(stored residual or None, y in 64 bits)."""
    v = x.float()
    out = None
    if r is not None:
        out = (v + r.float()).to(r.dtype)
        v = out.float()
    v = v.numpy().astype(np.float64)
    wt = w.float().numpy().astype(np.float64) + float(plus_one)
    return out, v / np.sqrt((v * v).mean(1, keepdims=True) + EPS) * wt


def on(t, dev):
    return None if t is None else t.to(dev)


def check_y(y, want):
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= np.abs(want) * (2.0 ** -8 + F32) + 2.0 ** -133).all(), err.max()


def check_y8(y8, scale, want):
    T, d = want.shape
    g = want.reshape(T, d // 64, 64)
    amax = np.abs(g).max(2)
    s = scale.cpu().numpy().astype(np.float64)
    assert (np.abs(s - amax / 448) <= amax / 448 * F32 + 2.0 ** -149).all()
    got = y8.float().cpu().numpy().astype(np.float64).reshape(g.shape) * s[:, :, None]
    bar = np.maximum(np.abs(g) * 2.0 ** -4, 2.0 ** -10 * s[:, :, None]) + 2 * F32 * np.abs(g)
    assert (np.abs(got - g) <= bar).all()


@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32],
                         ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rows_match_the_formula(dev, T, d, residual):
    plus_one = (T + d // 64) % 2 == 1
    x, w, r = inputs(T, d, residual, seed=T * 1000 + d, plus_one=plus_one)
    want_r, want = plain(x, w, r, plus_one)
    rout = None if r is None else torch.empty_like(r, device=dev)
    y = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    y, y8, scale = q4.add_norm(on(x, dev), on(w, dev), on(r, dev), eps=EPS, plus_one=plus_one,
                               residual_out=rout, y=y, e4m3=True)
    torch.cuda.synchronize()
    if r is not None:
        assert torch.equal(rout.cpu(), want_r)
    check_y(y, want)
    check_y8(y8, scale, want)


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_in_place_and_single_outputs(dev, residual):
    T, d = 9, 2112
    x, w, r = inputs(T, d, residual, seed=5)
    want_r, want = plain(x, w, r, False)
    xd, rd = on(x, dev), on(r, dev)
    y, y8, scale = q4.add_norm(xd, on(w, dev), rd, eps=EPS, residual_out=rd, y=xd)  # both in place
    assert y8 is None and scale is None and y is xd
    assert torch.equal(rd.cpu(), want_r)
    check_y(xd, want)
    # 8 bits alone, the residual's sum not stored: the inputs stay as they were
    xd, rd = on(x, dev), on(r, dev)
    y, y8, scale = q4.add_norm(xd, on(w, dev), rd, eps=EPS, e4m3=True)
    assert y is None
    check_y8(y8, scale, want)
    assert torch.equal(rd.cpu(), r) and torch.equal(xd.cpu(), x)


def test_zero_huge_and_non_finite_rows(dev):
    T, d = 6, 256
    x, w, _ = inputs(T, d, None, seed=6)
    x[0] = 0.0                      # y = 0, scale = 0
    x[1, 64:128] = 0.0              # one group of zeros
    x[2, 7] = float("nan")          # that row only
    x[3, 9] = float("inf")          # 0 everywhere else
    x[4] *= 1e-30                   # the square underflows: eps carries the root
    xd, wd = on(x, dev), on(w, dev)
    y, y8, scale = q4.add_norm(xd, wd, eps=EPS, y=torch.empty_like(xd), e4m3=True)
    y, y8, scale = y.float().cpu(), y8.float().cpu(), scale.cpu()
    assert (y[0] == 0).all() and (y8[0] == 0).all() and (scale[0] == 0).all()
    assert scale[1, 1] == 0 and (y8[1, 64:128] == 0).all() and (scale[1, [0, 2, 3]] > 0).all()
    assert y[2].isnan().all() and y8[2].isnan().all() and scale[2].isnan().all()
    assert y[3, 9].isnan() and (y[3, :9] == 0).all() and (y[3, 10:] == 0).all()
    assert y8[3, :64].isnan().all() and scale[3, 0].isnan() and (y8[3, 64:] == 0).all()
    keep = [1, 4, 5]
    _, want = plain(x[keep], w, None, False)
    check_y(y[keep].to(torch.bfloat16), want)


def test_another_stream_and_graph_replays(dev):
    T, d = 5, 2048
    x, w, r = inputs(T, d, torch.bfloat16, seed=8)
    xd, wd, rd = on(x, dev), on(w, dev), on(r, dev)
    want = q4.add_norm(xd, wd, rd, eps=EPS)[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(want)
    q4.add_norm(xd, wd, rd, eps=EPS, y=got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    # a captured step accumulates into the residual in place at every replay
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4.add_norm(xd, wd, rd, eps=EPS, residual_out=rd, y=y)
    rd.copy_(r)
    ref = rd.clone()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        yr = q4.add_norm(xd, wd, ref, eps=EPS, residual_out=ref)[0]
        assert torch.equal(rd, ref) and torch.equal(y, yr)
