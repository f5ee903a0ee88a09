"""Which bf16 products are exact, and what the others may lose: sums of large products that
cancel, with small ones next to them.  Products of fewer than 128 rows (of an expert, on
average) are exact.

In eight columns 8 i .. 8 i + 7 two products +p and -p, 2^17 <= p < 2^18, meet six small ones.
An exact product keeps the small ones to the bar of sums in fp32, (128 + blocks + 18) 2^-23 of
the sum S of all magnitudes (each of the additions off by at most 2^-23 of a partial sum), and
half a bf16 step of what remains.  A product that is cut at 2^-13 of the largest one's power of two,
here at 2^4, loses small products below 16 altogether: several times that bar."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain
from routings import device_routing, quantised_rows, selections, values

pytestmark = pytest.mark.gpu
f8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def bar_of(size, K):
    return (128 + -(-K // 128) + 18) * 2.0 ** -23 * size


def codes(v):
    c = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(f8)
    assert (c.float().numpy() == v).all()
    return c


def cancelling(rng, T, N, K, small, large=(384, 416, 448), apart=False):
    """x [T, K], w [N, K] (values): in one group of eight columns of every 128 (and of a last 64)
    two products that cancel; the other six, or with apart six of the group next to it, are of
    small[0] and small[1]."""
    x, w = np.zeros((T, K)), np.zeros((N, K))
    for b in range(0, K, 128):
        at = int(rng.integers(0, min(128, K - b) // 8))
        cols = b + 8 * at + rng.permutation(8)
        x[:, cols[:2]] = rng.choice(large, (T, 1))
        w[:, cols[0]] = rng.choice(large, N)
        w[:, cols[1]] = -w[:, cols[0]]
        if apart:
            cols = b + 8 * (at ^ 1) + rng.permutation(8)
        x[:, cols[2:]], w[:, cols[2:]] = rng.choice(small[0], (T, 6)), rng.choice(small[1], (N, 6))
    return x, w


FEW = ([2.5, 3, 3.5, 3.75],) * 2  # products of at most 14.1


def check(y, x, w, extra=0.0):
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
    bar = bar_of(size, x.shape[1]) + np.abs(want) * 2.0 ** -8 + extra
    worst = (err / bar).max()
    assert worst <= 1, worst


def linear(dev, x, w):
    (T, K), N = x.shape, w.shape[0]
    kb = -(-K // 128)
    return q4.linear_e4m3(codes(w).to(dev), torch.ones(-(-N // 128), kb, device=dev), codes(x).to(dev),
                          torch.ones(T, kb, device=dev))


# one token, decode batches, output heads, up to the last number of rows that is exact
EXACT = [(1, 2048, 64), (1, 16383, 64), (1, 16384, 64), (1, 40001, 192), (1, 140001, 64),
         (16, 16383, 64), (16, 16384, 192), (16, 40001, 64), (16, 140001, 64), (17, 5000, 192),
         (32, 4096, 64), (32, 4112, 64), (32, 32000, 64), (33, 257, 576), (64, 2050, 320),
         (64, 9000, 64), (64, 32000, 64), (65, 4100, 192), (100, 1100, 320), (127, 130, 640),
         (127, 4100, 64), (127, 8200, 64), (127, 40001, 64)]


@pytest.mark.parametrize("T,N,K", EXACT)
def test_fewer_than_128_tokens_lose_no_product(dev, T, N, K):
    x, w = cancelling(np.random.default_rng(T * 17 + N + K), T, N, K, FEW)
    check(linear(dev, x, w), x, w)


def experts(dev, rng, T, E, k, N, K, small, **how):
    """(rows a, b, y, x, w) of every expert that has rows."""
    idx, wt = selections(rng, T, E, k, 1.0)
    r, o = device_routing(idx, wt, E, dev)
    x, w = cancelling(rng, T * k, E * N, K, small, **how)
    w, kb = w.reshape(E, N, K), -(-K // 128)
    y = q4.experts_e4m3(codes(w).to(dev), torch.ones(E, -(-N // 128), kb, device=dev), codes(x).to(dev),
                        torch.ones(T * k, kb, device=dev), r)
    for e in range(E):
        a, b = int(o["offsets"][e]), int(o["offsets"][e + 1])
        if a < b:
            yield y[a:b], x[a:b], w[e]


@pytest.mark.parametrize("T,E,k,N,K", [(1, 8, 2, 300, 64), (60, 4, 2, 320, 192), (70, 4, 2, 300, 192),
                                       (400, 16, 4, 300, 320), (511, 16, 4, 257, 64)])
def test_experts_of_few_rows_lose_no_product(dev, T, E, k, N, K):
    for y, x, w in experts(dev, np.random.default_rng(T + N), T, E, k, N, K, FEW):
        check(y, x, w)


# the same bar for ordinary values and scales, whose factors xs * ws are rounded once
@pytest.mark.parametrize("T,N,K", [(1, 16500, 192), (16, 40001, 128), (17, 1000, 512), (33, 257, 576),
                                   (65, 4100, 256), (127, 130, 640), (127, 9000, 192)])
def test_ordinary_values_of_few_tokens(dev, T, N, K):
    rng = np.random.default_rng(T + N)
    x, xs = quantised_rows(rng, T, K)
    w, ws = q4.quantize_blocks(torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)))
    want, size = plain.product(values(w), ws.numpy(), values(x), xs.numpy())
    y = q4.linear_e4m3(w.to(dev), ws.to(dev), x.to(dev), xs.to(dev))
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bar_of(size, K) + np.abs(want) * 2.0 ** -8).all()


# every tile of the calls that may lose something
CUT = [(128, 130, 640), (128, 4100, 64), (200, 2050, 320), (200, 8200, 192), (300, 2050, 320),
       (2100, 2100, 192), (4100, 4100, 192)]


def pins(run):
    """What may be lost, and no more: run(small, **how) gives (y, x, w) of every matrix."""
    # bits from 2^-13 of the largest product on are kept: multiples of 8 next to 2^16
    for y, x, w in run(([2, 4], [4, 12, 20]), large=(256,)):
        check(y, x, w)
    # products of another group of eight columns are kept
    for y, x, w in run(FEW, apart=True):
        check(y, x, w)
    # each of six small products loses less than 2^4 (where the large ones lie below 2^18)
    for y, x, w in run(FEW):
        check(y, x, w, 6 * 16.0 * -(-x.shape[1] // 128))


@pytest.mark.parametrize("T,N,K", CUT)
def test_what_a_cut_product_loses(dev, T, N, K):
    rng = np.random.default_rng(T + N + K)

    def run(small, **how):
        x, w = cancelling(rng, T, N, K, small, **how)
        return [(linear(dev, x, w), x, w)]

    pins(run)


@pytest.mark.parametrize("T,E,k,N,K", [(512, 16, 4, 300, 320), (700, 8, 2, 257, 192)])
def test_what_a_cut_expert_product_loses(dev, T, E, k, N, K):
    rng = np.random.default_rng(T + N)
    pins(lambda small, **how: experts(dev, rng, T, E, k, N, K, small, **how))
