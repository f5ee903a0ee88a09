"""How exactly moe_linear adds, in each of its kernels.

Bar: a product of two bf16 values is exact in fp32; a row's sum is made of K / 32 matrix
instructions, taken as four roundings each (one per eight of a lane group's columns), and
20 joins.  A rounding is at most 2^-24 of the running sum, which stays within four
root-sums of squares R = sqrt(sum (w x)^2) of products of either sign:
    |err| <= (K / 8 + 20) * 2^-24 * 4 R.
The roundings' signs cancel, so the kernels reach a small part of it.  The test shows what
the bar tells apart: the rounding of the sums to bf16, and a single missing product.  Of
the products at K = 8192, where the bar is widest (R = 0.046 * 90, so 1.1e-3), one in 16
has the code 8, whose weight is 0 +- 0.001, and of the others, |w| = 0.01 j for j = 1 .. 8,
those with |x| below 0.11 / j, 3 % on average, are smaller: nine in ten are larger."""
import numpy as np
import pytest
import torch

import oracle
import q4_routed_expert_amd as q4
from workloads import bf16_bits, bits_to_f32, q4_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("N,K,T", [
    (300, 64, 3), (2048, 2048, 1), (333, 8192, 64), (4097, 576, 32), (6000, 2048, 17),   # split
    (8192, 2048, 5), (16384, 8192, 8), (20011, 1088, 16), (9001, 2112, 9),               # a pair of waves a tile
    (33000, 1024, 64), (40000, 960, 33), (33001, 2048, 8), (35000, 4096, 12),            # a wave a tile
    (9001, 8192, 64), (16400, 8128, 20), (8200, 4160, 64)])                              # x in chunks
def test_sums(dev, N, K, T):
    rng = np.random.default_rng(N + K + T)
    q, s, b = (m[0] for m in q4_matrix(rng, 1, N, K))
    x = bf16_bits(rng.standard_normal((T, K), dtype=np.float32))
    bf = lambda a: torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)   # noqa: E731
    args = torch.from_numpy(q.view(np.int32)).to(dev), bf(s), bf(b), bf(x)
    y = q4.linear(*args)
    yb = q4.linear(*args, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    rows = np.unique(np.r_[0:40, N // 2:N // 2 + 150, N - 60:N])
    w = (oracle.dequant(q[rows], s[rows], b[rows]).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    xf = bits_to_f32(x).astype(np.float64)
    want = xf @ w.T
    bar = (K / 8 + 20) * 2.0 ** -24 * 4 * np.sqrt((xf * xf) @ (w * w).T)
    got = y.cpu().numpy().astype(np.float64)[:, rows]
    assert (np.abs(got - want) <= bar).all(), (np.abs(got - want) / bar).max()
    # the bf16 output is the fp32 one rounded once
    assert torch.equal(yb, y.to(torch.bfloat16))
    # what the bar tells apart
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    assert (np.abs(rounded - want) > bar).mean() > 0.5
    products = np.abs(xf[:, None, :] * w[None, :20, :])
    assert (products > bar[:, :20, None]).mean() > 0.85
