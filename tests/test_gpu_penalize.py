"""penalize against its definition in 64 bits.

Bar, from the arithmetic: the division or product, frequency * n, two subtractions and one
addition per bias, each rounded once (2^-24 of a value that is at most the sum S of the
terms' magnitudes): (4 + biases of the token) 2^-24 S.  Tokens that nothing touches keep
their bits."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain

pytestmark = pytest.mark.gpu
f32, i32 = torch.float32, torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def words(allowed):
    """Bits [B, V] as int32 words; the bits behind V are ones and mean nothing."""
    B, V = allowed.shape
    bits = np.ones((B, -(-V // 32) * 32), np.uint8)
    bits[:, :V] = allowed
    return torch.from_numpy(np.packbits(bits, 1, bitorder="little").view(np.int32).copy())


def case(seed, B, V, L, n_bias, masked):
    rng = np.random.default_rng(seed)
    c = {"logits": (3 * rng.standard_normal((B, V))).astype(np.float32)}
    if L is not None:
        c["tokens"] = np.minimum((V * rng.random((B, L)) ** 5).astype(np.int32), V - 1)
        c["n_tokens"] = rng.integers(0, L + 1, B).astype(np.int32)
        c["n_tokens"][0] = L
        c["n_prompt"] = (c["n_tokens"] * rng.random(B)).astype(np.int32)
    for name, v in (("repetition", 1 + rng.random(B)), ("frequency", rng.standard_normal(B)),
                    ("presence", rng.standard_normal(B))):
        c[name] = v.astype(np.float32)
    if n_bias:
        c["bias_ids"] = rng.integers(-2, V + 2, (B, n_bias)).astype(np.int32)
        c["bias_ids"][:, ::3] = rng.integers(0, min(V, 4), (B, -(-n_bias // 3)))  # often the same
        c["bias"] = (4 * rng.standard_normal((B, n_bias))).astype(np.float32)
    if masked:
        c["allowed"] = rng.random((B, V)) >= masked
        if B > 1:
            c["allowed"][B - 1] = False
    return c


def call(c, dev, **kw):
    a = {n: torch.from_numpy(v).to(dev) for n, v in c.items() if n != "allowed"}
    if "allowed" in c:
        a["mask"] = words(c["allowed"]).to(dev)
    a.update(kw)
    return q4.penalize(a.pop("logits"), **a)


def check(c, got):
    got = got.cpu().numpy()
    for b in range(got.shape[0]):
        n = int(c["n_tokens"][b]) if "tokens" in c else 0
        ids = c["bias_ids"][b] if "bias_ids" in c else ()
        toks = c["tokens"][b, :n] if "tokens" in c else ()
        want, size = plain.penalize(
            c["logits"][b], toks, int(c["n_prompt"][b]) if "n_prompt" in c else 0, c["repetition"][b],
            c["frequency"][b], c["presence"][b], ids, c["bias"][b] if "bias" in c else (),
            c["allowed"][b] if "allowed" in c else None)
        V = want.size
        touched = np.zeros(V, np.int64)
        for v in ids:
            if 0 <= v < V:
                touched[v] += 1
        free = np.ones(V, bool)
        free[np.asarray(toks, np.int64)] = False
        free[touched > 0] = False
        ok = np.isfinite(want)
        assert np.array_equal(got[b][~ok], want[~ok].astype(np.float32))
        assert np.array_equal(got[b][free & ok], c["logits"][b][free & ok])
        assert (np.abs(got[b][ok] - want[ok]) <= ((4 + touched) * 2.0 ** -24 * size)[ok]).all()


SHAPES = [(1, 1, 1, 0, 0.0), (1, 33, 7, 3, 0.5), (2, 1000, 0, 5, 0.0), (3, 3001, 600, 20, 0.9),
          (5, 4096, 50, 0, 0.5), (4, 8195, 3000, 300, 0.99), (2, 50000, 20000, 7, 0.3),
          (1, 248320, 2000, 0, 0.0), (3, 70001, None, 1024, 0.5), (65, 2049, 90, 0, 0.2),
          (7, 30000, 400, 1, 0.0), (64, 20003, 100, 10, 0.7), (40, 220001, 9, 1000, 0.0),
          (2, 6000, 300, 1024, 0.0), (34, 248320, 33000, 9, 0.3),
          (11, 248319, 50, 5, 0.1)]


@pytest.mark.parametrize("B,V,L,n_bias,masked", SHAPES)
def test_rows_match_the_definition(dev, B, V, L, n_bias, masked):
    c = case(B * 1000 + V, B, V, L, n_bias, masked)
    room = torch.full((B + 1, V), 5.0, device=dev)
    got = call(c, dev, out=room)
    assert got is room and bool((room[B] == 5.0).all())
    check(c, room[:B])
    same = torch.from_numpy(c["logits"]).to(dev)
    out = call(c, dev, logits=same, out=same)  # in place
    assert out is same and torch.equal(same, room[:B])


def test_defaults_and_single_parameters(dev):
    c = case(1, 3, 900, 40, 0, 0.0)
    l, t = torch.from_numpy(c["logits"]).to(dev), torch.from_numpy(c["tokens"]).to(dev)
    assert torch.equal(q4.penalize(l), l)
    assert torch.equal(q4.penalize(l, tokens=t), l)
    a = q4.penalize(l, tokens=t, repetition=1.5, frequency=0.25, presence=-0.5)
    full = lambda v: torch.full((3,), v, device=dev)                                 # noqa: E731
    b = q4.penalize(l, tokens=t, repetition=full(1.5), frequency=full(0.25), presence=full(-0.5),
                    n_tokens=torch.full((3,), 40, dtype=i32, device=dev),
                    n_prompt=torch.full((3,), -7, dtype=i32, device=dev))
    assert torch.equal(a, b) and not torch.equal(a, l)
    # counts beyond the array, a prompt beyond the tokens, repetitions that are off
    n = torch.tensor([1 << 30, 40, -3], dtype=i32, device=dev)
    d = q4.penalize(l, tokens=t, n_tokens=n, frequency=1.0)
    e = q4.penalize(l, tokens=t, frequency=1.0)
    assert torch.equal(d[:2], e[:2]) and torch.equal(d[2], l[2])
    p = torch.full((3,), 41, dtype=i32, device=dev)
    assert torch.equal(q4.penalize(l, tokens=t, n_prompt=p, frequency=1.0, presence=1.0), l)
    off = torch.tensor([0.0, -2.0, float("nan")], device=dev)
    assert torch.equal(q4.penalize(l, tokens=t, repetition=off), l)


def test_non_finite_logits(dev):
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[inf, -inf, nan, 2.0, -2.0, 0.0]], device=dev)
    t = torch.arange(6, dtype=i32, device=dev).view(1, 6)
    y = q4.penalize(l, tokens=t, repetition=2.0, presence=1.0).cpu()[0]
    assert y[0] == inf and y[1] == -inf and y[2].isnan()
    assert y[3:].tolist() == [0.0, -5.0, -1.0]
    m = torch.zeros(1, 1, dtype=i32, device=dev)  # nothing allowed, a NaN is masked too
    y = q4.penalize(l, tokens=t, mask=m)
    assert bool((y == -inf).all())
    token, prob, _ = q4.sample(y, torch.full((1,), 0.5, device=dev))
    assert int(token) == 0 and float(prob) == 0.0


def test_padding_and_a_long_repeat(dev):
    # ids that are no tokens are passed over; one token 20000 times counts exactly
    B, V, L = 2, 5000, 20000
    t = torch.full((B, L), 4999, dtype=i32, device=dev)
    t[1] = torch.tensor([-1, V, -(1 << 31), (1 << 31) - 1], dtype=i32).repeat(L // 4).to(dev)
    l = torch.randn(B, V, device=dev)
    y = q4.penalize(l, tokens=t, frequency=0.5, presence=2.0, repetition=3.0)
    want = l[0, 4999] / 3.0 if l[0, 4999] > 0 else l[0, 4999] * 3.0
    assert abs(float(y[0, 4999]) - (float(want) - 10002.0)) <= 4 * 2.0 ** -24 * 10010
    assert torch.equal(y[0, :4999], l[0, :4999]) and torch.equal(y[1], l[1])


def test_biases_of_one_token_add_in_list_order(dev):
    B, V, n = 2, 40000, 200
    rng = np.random.default_rng(9)
    b = (1000 * rng.standard_normal((B, n))).astype(np.float32)
    ids = torch.full((B, n), V - 1, dtype=i32)
    l = torch.zeros(B, V)
    y = q4.penalize(l.to(dev), bias_ids=ids.to(dev), bias=torch.from_numpy(b).to(dev)).cpu()
    for r in range(B):
        s = np.float32(0.0)
        for v in b[r]:
            s = np.float32(s + v)
        assert y[r, V - 1] == s


def test_logits_past_32_bits(dev):
    # 2^32 bytes of logits: a row in the middle and the last one, the others as they were
    B, V, L = 1024, 1048576, 64
    l = torch.randn(B, V, device=dev)
    c = case(17, 2, V, L, 12, 0.3)
    c["allowed"][1] = c["allowed"][0][::-1]
    rows = [B // 2, B - 1]
    c["logits"] = l[rows].cpu().numpy()
    a = {n: torch.zeros((B,) + v.shape[1:], dtype=torch.from_numpy(v).dtype, device=dev)
         for n, v in c.items() if n not in ("logits", "allowed")}
    for n, t in a.items():
        t[rows] = torch.from_numpy(c[n]).to(dev)
    a["repetition"][a["repetition"] == 0] = 1.0
    a["mask"] = torch.full((B, V // 32), -1, dtype=i32, device=dev)
    a["mask"][rows] = words(c["allowed"]).to(dev)
    y = q4.penalize(l, **a)
    check(c, y[rows])
    others = [0, 1, B // 2 - 1, B // 2 + 1, B - 2]
    assert torch.equal(y[others], l[others])
    q4.penalize(l, out=l, **a)
    assert torch.equal(y, l)


def test_streams_and_graphs(dev):
    c = case(3, 4, 30011, 500, 30, 0.5)
    want = call(c, dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = {n: torch.from_numpy(v).to(dev) for n, v in c.items() if n != "allowed"}
    a["mask"] = words(c["allowed"]).to(dev)
    l = a.pop("logits")
    torch.cuda.synchronize()
    got = q4.penalize(l, stream=side, **a)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q4.penalize(l, **a)
    for i in range(3):
        l.mul_(-1.5)
        a["tokens"].sub_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q4.penalize(l, **a)), i
