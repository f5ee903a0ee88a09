"""The probability that moe_sample returns, for tokens far below the largest.

u = 0 draws the first kept token with a weight, so a row whose token 0 lies at a chosen
depth returns that token.  Bar: half an fp32 step, 2^-24 relative, plus the rounding of
the kept weights to multiples of 2^-43 of the largest (V 2^-44 of their sum at most) and
2^-43 for the 64-bit exponential.  All of it is relative to the probability itself."""
import math

import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4

pytestmark = pytest.mark.gpu
DEPTHS = np.concatenate([np.linspace(0.0, 30.3, 90), [14.0, 16.0, 20.0, 24.0, 28.0, 30.39]]).astype(np.float32)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def rows(V, temperature, seed):
    rng = np.random.default_rng(seed)
    l = np.full((DEPTHS.size, V), -np.inf, np.float32)
    l[:, 0] = -DEPTHS * np.float32(temperature)
    if V > 2:  # neighbours around and below the token, and the largest somewhere behind it
        l[:, 2:] = -np.abs(8 * rng.standard_normal((DEPTHS.size, V - 2))).astype(np.float32)
    l[:, V - 1] = 0.0
    return l


@pytest.mark.parametrize("V", [2, 700, 8192, 8193, 20000])
@pytest.mark.parametrize("temperature,kw", [(1.0, {}), (0.7, {}), (1.0, dict(top_k=1 << 15)),
                                            (1.3, dict(min_p=1e-14))], ids=["t1", "t0.7", "top_k", "min_p"])
def test_deep_tokens(dev, V, temperature, kw):
    l = rows(V, temperature, V)
    token, prob, _ = q4.sample(torch.from_numpy(l).to(dev), torch.zeros(len(l), device=dev),
                               temperature=temperature, **kw)
    torch.cuda.synchronize()
    assert (token == 0).all()
    t = float(np.float32(temperature))
    for b, p in enumerate(prob.cpu().numpy().astype(np.float64)):
        x = -l[b].astype(np.float64) / t
        want = math.exp(-x[0]) / math.fsum(np.exp(-x))
        assert abs(p - want) <= want * (2.0 ** -24 + V * 2.0 ** -44 + 2.0 ** -43), (DEPTHS[b], p, want)


def test_tokens_below_the_range_are_not_drawn(dev):
    for V in (3, 9000):
        l = np.full((1, V), -31.0, np.float32)
        l[0, V - 1] = 0.0
        token, prob, _ = q4.sample(torch.from_numpy(l).to(dev), torch.zeros(1, device=dev))
        assert int(token[0]) == V - 1 and float(prob[0]) == 1.0
