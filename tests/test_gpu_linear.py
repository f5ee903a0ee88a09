"""moe_linear against the products in 64 bits.

Bar: the products of bf16 values are exact in fp32; K of them are added in fp32
in some order, so |err| <= K * 2^-24 * sum_k |w x| in the worst case; the sums
run over at most K / 32 dependent additions of 32-term blocks and a few joins, and
errors of either sign cancel: 8 * sqrt(K) * 2^-24 * sum |w x| is far above what
they reach and far below one wrong or missing product (about sum |w x| / K).  A
bf16 output adds half a step, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain
from workloads import bf16_bits, bits_to_f32, q4_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(N, K, T, seed=0):
    rng = np.random.default_rng(seed)
    q, s, b = (m[0] for m in q4_matrix(rng, 1, N, K))
    return q, s, b, bf16_bits(rng.standard_normal((T, K), dtype=np.float32))


def put(dev, q, s, b, x):
    bf = lambda a: torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)  # noqa: E731
    return torch.from_numpy(q.view(np.int32)).to(dev), bf(s), bf(b), bf(x)


def check(y, q, s, b, x, rows=None):
    rows = np.arange(q.shape[0]) if rows is None else rows
    xf = bits_to_f32(x).astype(np.float64)
    want = plain.linear(q[rows], s[rows], b[rows], xf)
    K = xf.shape[1]
    # weights lie within 8.1 scales of 0, scales below 0.0151: sum |w x| <= 0.13 sum |x|;
    # a typical weight is half of that, so this is no more than twice the sum
    total = 0.13 * np.abs(xf).sum(1)[:, None]
    bar = 8 * np.sqrt(K) * 2.0 ** -24 * total
    if y.dtype == torch.bfloat16:
        bar = bar + np.abs(want) * 2.0 ** -8
    got = y.float().cpu().numpy().astype(np.float64)[:, rows]
    assert (np.abs(got - want) <= bar).all(), np.abs(got - want).max()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,K,T", [
    (1, 64, 1), (16, 64, 1), (17, 128, 3), (5, 192, 64), (100, 448, 16), (513, 512, 17),
    (2048, 2048, 1), (2049, 2048, 8), (1000, 4160, 5), (64, 8192, 33), (333, 8192, 64),
    (4097, 576, 32), (7000, 1024, 48), (30000, 256, 2), (9001, 2112, 9), (6000, 2048, 64),
    (16500, 640, 31), (300, 8128, 2),
    (20011, 64, 5), (17001, 192, 40), (16400, 4160, 20), (33000, 1088, 64), (40000, 448, 12),
    (16384, 8192, 8), (35000, 2112, 33)])
def test_products(dev, N, K, T, out):
    q, s, b, x = make(N, K, T, seed=N + K + T)
    y = q4.linear(*put(dev, q, s, b, x), out_dtype=out)
    torch.cuda.synchronize()
    assert y.shape == (T, N) and y.dtype == out
    check(y, q, s, b, x)


def test_rows_do_not_depend_on_each_other(dev):
    # every row alone gives the same bits as the batch, whatever else the batch holds
    for N, K, T in ((77, 192, 64), (5000, 2048, 37), (40000, 512, 16)):
        q, s, b, x = make(N, K, T, seed=N)
        qd, sd, bd, xd = put(dev, q, s, b, x)
        y = q4.linear(qd, sd, bd, xd)
        for t in (0, 1, T // 2, T - 1):
            assert torch.equal(q4.linear(qd, sd, bd, xd[t:t + 1].clone()), y[t:t + 1])
        xd2 = xd.clone()
        xd2[0] = float("nan")
        xd2[T - 1, 3] = float("inf")
        y2 = q4.linear(qd, sd, bd, xd2)
        assert torch.equal(y2[1:T - 1], y[1:T - 1])
        assert y2[0].isnan().all() and not y2[T - 1].isfinite().any()


def test_written_range(dev):
    # the elements behind y stay as they were, for row lengths of every alignment
    for N in (15, 16, 17, 18, 4099):
        q, s, b, x = make(N, 320, 3, seed=N)
        for out in (torch.float32, torch.bfloat16):
            buf = torch.full((3 * N + 64,), 7.0, dtype=out, device=dev)
            q4.linear(*put(dev, q, s, b, x), out_dtype=out, y=buf)
            torch.cuda.synchronize()
            assert (buf[3 * N:] == 7.0).all()
            check(buf[:3 * N].view(3, N), q, s, b, x)


def test_widest_matrix_passes_32_bit_offsets(dev):
    # 2^20 rows of 8192 columns: 4 GiB of codes; the rows at the far end are checked
    N, K, T = q4._abi.MOE_MAX_VOCAB, 8192, 2
    g = torch.Generator(device=dev).manual_seed(3)
    q = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device=dev, dtype=torch.int32)
    s = (0.005 + 0.01 * torch.rand(N, K // 64, generator=g, device=dev)).to(torch.bfloat16)
    b = (-8.0 * s.float()).to(torch.bfloat16)
    x = torch.randn(T, K, generator=g, device=dev).to(torch.bfloat16)
    y = q4.linear(q, s, b, x)
    rows = np.r_[0:20, N // 2 - 10:N // 2 + 10, N - 40:N]
    sub = torch.from_numpy(rows).to(dev)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)              # noqa: E731
    check(y[:, sub], q[sub].cpu().numpy().view(np.uint32), bits(s[sub]), bits(b[sub]), bits(x))


def test_graph_replays_and_streams(dev):
    N, K, T = 3000, 2048, 6
    q, s, b, x = make(N, K, T, seed=1)
    qd, sd, bd, xd = put(dev, q, s, b, x)
    want = q4.linear(qd, sd, bd, xd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    q4.linear(qd, sd, bd, xd, y=y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4.linear(qd, sd, bd, xd, y=y)
    for rep in range(3):
        xd.copy_(torch.randn(T, K, device=dev).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, q4.linear(qd, sd, bd, xd))
