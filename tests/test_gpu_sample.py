"""moe_sample against the definition with exact integer weights.

Bars: tokens exact.  The kernel's weights and the oracle's are the same rounding of
exp in 64 bits (2^-52 relative) to multiples of 2^-43, so they differ by one unit in
about one weight of 2^9; a token can then differ only where u or top_p falls within
V units of a border, less than 2^20 * 2^-43 = 2^-23 of the sum in the worst case and
about 2^-35 for V = 10^5, where the differences have either sign.  prob: one fp32 rounding,
2^-24 relative, plus 2^-30.
"""
import numpy as np
import pytest
import torch

import oracle
import q4_routed_expert_amd as q4
from oracle import operators as plain
from workloads import random_lm

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def logits_for(B, V, seed, coarse=False, spread=2.0):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((B, V))).astype(np.float32)
    for b in range(B):
        l[b, rng.integers(0, V, 6)] += np.float32(3 * spread)
    return np.round(l * 8) / np.float32(8) if coarse else l


def check(dev, l, u, temperature, top_k, top_p, min_p, arrays=True, stream=None, ws=None):
    l = np.ascontiguousarray(l, np.float32)
    B, V = l.shape
    full = lambda v, t: np.full(B, v, t) if np.isscalar(v) else np.asarray(v, t)   # noqa: E731
    u, tt = full(u, np.float32), full(temperature, np.float32)
    kk, pp, mm = full(top_k, np.int32), full(top_p, np.float32), full(min_p, np.float32)
    put = lambda a: torch.from_numpy(a).to(dev)                                     # noqa: E731
    if arrays:
        kw = dict(temperature=put(tt), top_k=put(kk), top_p=put(pp), min_p=put(mm))
    else:
        kw = dict(temperature=float(tt[0]), top_k=int(kk[0]), top_p=float(pp[0]), min_p=float(mm[0]))
    token, prob, _ = q4.sample(put(l), put(u), ws=ws, stream=stream, **kw)
    torch.cuda.synchronize()
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    for b in range(B):
        par = (tt[b], kk[b], pp[b], mm[b])
        want, wp = plain.sample(l[b], u[b], *par)
        assert token[b] == want, (b, u[b], par, token[b], want)
        assert abs(prob[b] - wp) <= wp * 2.0 ** -24 + 2.0 ** -30, (b, prob[b], wp)


SIZES = [(1, 1), (3, 2), (2, 63), (5, 1000), (4, 2047), (4, 2048), (4, 2049), (37, 3001),
         (2, 4097), (3, 8191), (2, 8192), (2, 8193), (2, 16385), (7, 30011), (1, 248320), (3, 100003)]
FILTERS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.05),
           (0.8, 40, 0.95, 0.02), (0.0, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.0), (2.5, 1000, 0.3, 0.0),
           (5.0, 0, 0.999, 0.0), (1.0, 0, 0.0, 0.0), (0.6, 0, 0.5, 1.0), (50.0, 700, 0.99, 0.5)]


@pytest.mark.parametrize("coarse", [False, True], ids=["fine", "coarse"])
@pytest.mark.parametrize("B,V", SIZES)
def test_tokens_are_exact(dev, B, V, coarse):
    rng = np.random.default_rng(V + B)
    l = logits_for(B, V, V, coarse)
    for f in FILTERS:
        check(dev, l, rng.random(B).astype(np.float32), *f)


def test_rows_have_their_own_parameters(dev):
    B, V = len(FILTERS), 5003
    l = logits_for(B, V, 1)
    rng = np.random.default_rng(1)
    t, k, p, m = (np.array(c) for c in zip(*FILTERS))
    for _ in range(5):
        check(dev, l, rng.random(B).astype(np.float32), t, k, p, m)
    check(dev, l, 0.25, 0.8, 40, 0.95, 0.02, arrays=False)


def test_edges_of_u(dev):
    l = logits_for(6, 4000, 2)
    u = np.array([0.0, 1.0, 1.0 - 2.0 ** -24, -3.0, 7.5, NAN], np.float32)
    for f in FILTERS:
        put = lambda a: torch.from_numpy(np.asarray(a)).to(dev)                     # noqa: E731
        token, _, _ = q4.sample(put(l), put(u), *f)
        token = token.cpu().numpy()
        for b in range(6):
            want, _ = plain.sample(l[b], 0.0 if u[b] != u[b] else u[b], *f)
            assert token[b] == want, (b, f)


def test_masks_ties_and_empty_rows(dev):
    V, low = 9000, -np.finfo(np.float32).max
    l = np.stack([logits_for(1, V, 30 + b)[0] for b in range(14)])
    rng = np.random.default_rng(5)
    l[0] = -INF                                   # nothing left: token 0, prob 0
    l[1] = NAN
    l[2] = low                                    # the mask's lowest value everywhere: uniform
    l[3] = -INF
    l[3, 8999] = -5.0                             # one live token, the last
    l[4, rng.random(V) < 0.99] = -INF
    l[5, rng.random(V) < 0.5] = NAN
    l[6, [17, 4000]] = INF                        # two infinities share everything
    l[7] = 0.0
    l[7, ::2] = -0.0                              # equal
    l[8] = 3.0                                    # all equal: more ties than the list holds
    l[9, : V // 2] = np.float32(l[9].max())
    l[10, rng.random(V) < 0.9] = low
    l[11] = np.where(np.arange(V) % 2 == 0, 1.0, 1.0 + 2.0 ** -23)
    l[12] *= 1e30
    l[13] *= 1e-30
    for f in FILTERS + [(1.0, 5000, 1.0, 0.0), (1.0, 4097, 0.5, 0.0), (1.0, 0, 0.6, 0.0),
                        (INF, 0, 1.0, 0.0), (INF, 4500, 0.75, 0.0), (1e-30, 0, 0.5, 0.0),
                        (NAN, 3, 0.5, 0.0), (1.0, -4, NAN, NAN)]:
        u = (rng.random(14) * 0.998 + 0.001).astype(np.float32)
        p = 1.0 if f[2] != f[2] else f[2]
        m = 0.0 if f[3] != f[3] else f[3]
        got = q4.sample(torch.from_numpy(l).to(dev), torch.from_numpy(u).to(dev), *f)[0].cpu().numpy()
        for b in range(14):
            want, _ = plain.sample(l[b], u[b], f[0], f[1], p, m)
            assert got[b] == want, (b, f, u[b], got[b], want)


def test_largest_vocabulary_and_batch(dev):
    V = q4._abi.MOE_MAX_VOCAB
    l = logits_for(2, V, 77)
    l[1] = np.round(l[1])                         # tens of thousands of equal logits
    for f in ((1.0, 0, 0.95, 0.0), (0.9, 0, 1.0, 0.0), (1.0, 60000, 0.9, 0.0)):
        check(dev, l, np.array([0.3, 0.7], np.float32), *f)
    B = q4._abi.MOE_MAX_SAMPLE_ROWS
    l = logits_for(B, 257, 78)
    check(dev, l, np.random.default_rng(1).random(B).astype(np.float32), 1.0, 20, 0.9, 0.01)


def test_draws_follow_the_weights(dev):
    # a fine grid of u hits every token in proportion to its weight, in index order
    l = np.log(np.array([[1, 2, 3, 4, 6]], np.float32))
    n = 1600
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    token, prob, _ = q4.sample(torch.from_numpy(np.repeat(l, 1000, 0)).to(dev),
                               torch.from_numpy(u[:1000]).to(dev))
    rest, _, _ = q4.sample(torch.from_numpy(np.repeat(l, 600, 0)).to(dev),
                           torch.from_numpy(u[1000:]).to(dev))
    t = np.concatenate([token.cpu().numpy(), rest.cpu().numpy()])
    assert np.bincount(t).tolist() == [100, 200, 300, 400, 600] and (np.diff(t) >= 0).all()


def test_given_buffers_embedding_rows_and_alignment(dev):
    V, d, B = 777, 320, 5
    x, head, embed = random_lm(np.random.default_rng(3), V, d)
    lm = q4.DeviceLmHead.from_host(head, embed, dev)
    l = logits_for(B, V, 3)
    u = np.linspace(0.05, 0.95, B).astype(np.float32)
    token = torch.full((B + 3,), -7, dtype=torch.int32, device=dev)
    prob = torch.full((B + 3,), -7.0, device=dev)
    xn = torch.zeros(B + 1, d, dtype=torch.bfloat16, device=dev)
    par = torch.zeros(B + 1, device=dev)
    par[1:] = 0.8
    t, p, n = q4.sample(torch.from_numpy(l).to(dev), torch.from_numpy(u).to(dev), top_k=30, lm=lm,
                        temperature=par[1:], token=token[1:], prob=prob[1:], x_next=xn)
    torch.cuda.synchronize()
    assert token[0] == -7 and (token[B + 1:] == -7).all() and (prob[B + 1:] == -7.0).all()
    assert (xn[B] == 0).all()
    for b in range(B):
        want, _ = plain.sample(l[b], u[b], np.float32(0.8), 30)
        assert int(t[b]) == want
        row = oracle.embed_row(embed["q"], embed["scale"], embed["bias"], want)
        assert np.array_equal(xn[b].view(torch.int16).cpu().numpy().view(np.uint16), row)


def test_batches_streams_and_graphs_agree(dev):
    # a row's token does not depend on its batch; two streams with a workspace each;
    # replays of a captured call with new inputs
    B, V = 20, 40000
    l = torch.from_numpy(logits_for(B, V, 9)).to(dev)
    u = torch.rand(B, device=dev)
    par = dict(temperature=0.9, top_k=300, top_p=0.9, min_p=0.001)
    want, wp, _ = q4.sample(l, u, **par)
    for b in (0, 7, B - 1):
        t, p, _ = q4.sample(l[b:b + 1].clone(), u[b:b + 1].clone(), **par)
        assert torch.equal(t, want[b:b + 1]) and torch.equal(p, wp[b:b + 1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    ws = [q4.sample_workspace(B, V, dev) for _ in streams]
    outs = []
    for rep in range(4):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                outs.append(q4.sample(l, u, ws=w, stream=s, **par)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    token, prob = torch.empty_like(want), torch.empty_like(wp)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4.sample(l, u, token=token, prob=prob, ws=ws[0], **par)
    for rep in range(3):
        l.copy_(torch.from_numpy(logits_for(B, V, 100 + rep, coarse=rep == 1)))
        u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        t, p, _ = q4.sample(l, u, ws=ws[1], **par)
        assert torch.equal(token, t) and torch.equal(prob, p)
