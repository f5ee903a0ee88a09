"""The 8-bit output of moe_add_norm at its borders: y8 = e4m3(y / scale) with the
stored scale, for values next to a rounding border, for groups of tiny values and
for groups with an infinity.

Rows of +-1 have the mean square 1, so with eps = 0 and no residual y is the weight
itself, up to its sign: scale and codes then follow from the weight in fp32 without
any tolerance.  With other rows y carries an error of 2^-17 relative (the bar of the
operator's other tests), and a subnormal scale is off by up to 2^-150, which moves a
value of 448 scales by 448 times that.
"""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -17


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def codes(z):
    """Values of e4m3 codes, nearest even, of fp32 numbers within +-448."""
    return torch.from_numpy(np.clip(z, -448, 448)).to(torch.float8_e4m3fn).float().numpy()


def quantised(dev, x, w, **kw):
    _, y8, scale = q4.add_norm(x.to(dev), w.to(dev), e4m3=True, **kw)
    torch.cuda.synchronize()
    return y8.float().cpu().numpy(), scale.cpu().numpy()


def test_codes_are_the_quotient_by_the_stored_scale(dev):
    d, other = 8192, 0
    rng = np.random.default_rng(11)
    for rep in range(12):
        x = torch.from_numpy(rng.choice([-1.0, 1.0], (2, d))).to(torch.bfloat16)
        w = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(torch.bfloat16)
        y = (x.float() * w.float()).numpy().reshape(2, -1, 64)
        amax = np.abs(y).max(2, keepdims=True)
        s = amax / np.float32(448)
        want = codes(y / s)
        # the inputs tell the quotient from a factor 448 / max|y|
        other += int((want != codes(y * (np.float32(448) / amax))).sum())
        y8, scale = quantised(dev, x, w, eps=0.0)
        assert np.array_equal(scale, s[:, :, 0])
        assert np.array_equal(y8.reshape(want.shape), want), rep
    assert other > 0


def test_groups_of_tiny_values(dev):
    # weights of every size down to bf16's smallest, 2^-133, a group each
    d = 64 * 64
    rng = np.random.default_rng(12)
    size = 2.0 ** np.linspace(-133, -90, 64)
    w = torch.from_numpy((size[:, None] * rng.uniform(0.25, 1.0, (64, 64))).reshape(-1)).to(torch.bfloat16)
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (1, d))).to(torch.bfloat16)
    y = (x.float() * w.float()).numpy().reshape(64, 64)
    s = np.abs(y).max(1) / np.float32(448)
    y8, scale = quantised(dev, x, w, eps=0.0)
    assert np.array_equal(scale[0], s)
    with np.errstate(divide="ignore", invalid="ignore"):
        want = np.where(s[:, None] > 0, codes(y / s[:, None]), 0.0)
    assert np.array_equal(y8.reshape(64, 64), want)
    # rows whose own values are tiny, down to scales that are 0
    x = torch.ones(64, d)
    x[:, :64] = torch.from_numpy(2.0 ** -np.linspace(90, 133, 64))[:, None]
    x[:, 5:64:2] *= 0.5
    x = x.to(torch.bfloat16)
    w = torch.full((d,), 2.0 ** -12, dtype=torch.bfloat16)
    y8, scale = quantised(dev, x, w, eps=1e-6)
    v = x.double().numpy()
    y = (v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * 2.0 ** -12)[:, :64]
    s = scale[:, 0].astype(np.float64)
    amax = np.abs(y).max(1)
    assert (np.abs(s - amax / 448) <= amax / 448 * F32 + 2.0 ** -149).all()
    assert (s == 0).any() and (s > 0).any()
    bar = np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10 * s[:, None]) + 2 * F32 * np.abs(y) + 448 * 2.0 ** -149
    assert (np.abs(y8[:, :64] * s[:, None] - y) <= bar).all()
    assert (y8[s == 0, :64] == 0).all()


def test_groups_with_an_infinity(dev):
    x = torch.ones(1, 256, dtype=torch.bfloat16)
    x[0, 70] = 4.0  # times 3e38: past fp32's range
    w = torch.full((256,), 3e38, dtype=torch.bfloat16)
    w[:64] = 1.0
    y8, scale = quantised(dev, x, w, eps=0.0)
    assert np.isinf(scale[0, 1]) and np.isfinite(scale[0, [0, 2, 3]]).all()
    assert np.isnan(y8[0, 70]) and (np.delete(y8[0, 64:128], 6) == 0).all()
    assert (y8[0, :64] == 448).all() and (y8[0, 128:] == 448).all()
