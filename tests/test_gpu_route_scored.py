"""moe_route_scored, and decoding from a given selection, against the definition
in 64 bits.

Bars: selections, counts, permutations and maps exact (scores are compared in 64
bits on both sides; the inputs' scores differ by far more than 1e-15 or are
equal); weights within 2^-24 relative (one rounding to fp32) plus 1e-12 for the
64-bit arithmetic.
"""
import numpy as np
import pytest
import torch

import oracle
import q4_routed_expert_amd as q4
from oracle import operators as plain
from workloads import bits_to_f32, random_layer, random_x

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def small_layer(E, k, dev):
    return q4.DeviceLayer.from_host(random_layer(np.random.default_rng(0), 64, 64, E, k), dev)


def run(dev, logits, k, balance=None, layer=None, **kw):
    T, E = logits.shape
    layer = layer or small_layer(E, k, dev)
    r = q4.DeviceRouting(T, E, k, dev)
    r.logits.copy_(torch.from_numpy(np.ascontiguousarray(logits, np.float32)))
    b = None if balance is None else torch.from_numpy(np.asarray(balance, np.float32)).to(dev)
    q4.route_scored(layer, None, q4.RouterSpec(balance=b, **kw), r, logits_in=True)
    torch.cuda.synchronize()
    return r


def check(r, logits, k, balance=None, **kw):
    E = logits.shape[1]
    idx, w = plain.route_scored(logits, k, balance=balance, **kw)
    assert np.array_equal(r.topk_idx.cpu().numpy(), idx)
    got = r.topk_w.cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= np.abs(w) * 2.0 ** -24 + 1e-12 * abs(kw.get("scale", 1.0))).all()
    want = plain.sort_assignments(idx, E)
    for name in ("counts", "offsets", "perm", "inv_perm"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), want[name]), name
    for rows, m, n in ((32, r.block_map, r.n_blocks), (128, r.tile_map, r.n_tiles)):
        t = plain.tiles(want["counts"], rows)
        assert int(n.cpu()[0]) == len(t)
        assert np.array_equal(m.cpu().numpy()[:len(t)], t)


CASES = [
    # T, E, k, kw
    (1, 256, 8, dict(score="sigmoid", n_groups=8, top_groups=4, group_top=2, scale=2.5)),
    (1, 1, 1, dict()),
    (3, 6, 2, dict(score="sigmoid", n_groups=3, top_groups=2, group_top=2)),
    (257, 160, 6, dict(n_groups=8, top_groups=3, group_top=1, renorm=False, scale=16.0)),
    (64, 256, 8, dict(score="softmax")),
    (65, 130, 7, dict(score="sigmoid", renorm=False)),
    (33, 64, 8, dict(score="sigmoid", n_groups=64, top_groups=8, group_top=1)),
    (300, 48, 5, dict(score="softmax", n_groups=4, top_groups=4, group_top=2)),
    (129, 252, 8, dict(score="sigmoid", n_groups=2, top_groups=1, group_top=2)),
    (1025, 32, 4, dict(score="softmax", n_groups=8, top_groups=1, group_top=2)),
    (17, 256, 8, dict(score="sigmoid", n_groups=1, scale=-0.5)),
    (16, 256, 8, dict(score="sigmoid", n_groups=16, top_groups=5, group_top=2)),
    (15, 200, 3, dict(score="softmax", n_groups=50, top_groups=2, group_top=2)),
    (2, 128, 8, dict(score="sigmoid", n_groups=1)),
    (9, 256, 8, dict(score="softmax", n_groups=2, top_groups=1, group_top=2, renorm=False)),
    (600, 64, 8, dict(score="softmax", n_groups=16, top_groups=4, group_top=2)),
]


@pytest.mark.parametrize("with_balance", [False, True], ids=["plain", "balance"])
@pytest.mark.parametrize("T,E,k,kw", CASES, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_random_scores(dev, T, E, k, kw, with_balance):
    rng = np.random.default_rng(T * 7 + E)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    b = (0.2 * rng.standard_normal(E)).astype(np.float32) if with_balance else None
    check(run(dev, logits, k, b, **kw), logits, k, b, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(n_groups=4, top_groups=2, group_top=2),
                                    dict(n_groups=16, top_groups=9, group_top=1)],
                         ids=["flat", "4of2", "16of9"])
def test_ties_masks_and_empty_rows(dev, score, groups):
    T, E, k = 40, 64, 8
    rng = np.random.default_rng(3)
    l = np.round(rng.standard_normal((T, E)) * 2).astype(np.float32) / 2  # many equal scores
    l[0] = 0.0
    l[1] = -0.0
    l[1, ::3] = 0.0
    l[2] = -INF                       # a row that its mask leaves empty
    l[3] = NAN
    l[4] = -np.finfo(np.float32).max  # masked with the lowest value: all equal
    l[5, : E - 3] = -INF              # fewer live experts than slots
    l[6, 10] = INF
    l[7, [5, 50]] = INF
    l[8, ::2] = NAN
    l[9, 1:] = -np.finfo(np.float32).max
    l[10] = 30.0 + np.arange(E, dtype=np.float32)[::-1] * 0.01 if score == "softmax" else 1.0
    for b in (None, np.where(np.arange(E) % 5 == 0, -INF, 0.25).astype(np.float32),
              np.full(E, NAN, np.float32)):
        kw = dict(score=score, **groups)
        check(run(dev, l, k, b, **kw), l, k, b, **kw)


def test_longest_chunk(dev):
    T, E, k = q4._abi.MOE_MAX_TOKENS, 256, 8
    rng = np.random.default_rng(9)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=8, top_groups=4, group_top=2, scale=2.5)
    r = run(dev, logits, k, b, **kw)
    sub = np.concatenate([np.arange(40), rng.integers(0, T, 200), np.arange(T - 40, T)])
    idx, w = plain.route_scored(logits[sub], k, balance=b, **kw)
    got = r.topk_idx.cpu().numpy()
    assert np.array_equal(got[sub], idx)
    want = plain.sort_assignments(got, E)  # the sorted order of every selection
    for name in ("counts", "offsets", "perm", "inv_perm"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), want[name]), name


@pytest.mark.parametrize("T", [1, 3, 8, 16, 70])
def test_the_experts_products_follow_the_selection(dev, T):
    # x -> scored routing -> prefill, and the same selection through decode: both
    # against the oracle's layer with that selection (the bar of the layer's own
    # parity tests: 2e-2 RMS, or half a bf16 step + 2e-3 RMS for large values)
    rng = np.random.default_rng(70 + T)
    L = random_layer(rng, 256, 128, 32, 4, router_bias=True)
    x = random_x(rng, T, 256)
    layer = q4.DeviceLayer.from_host(L, dev)
    xd = torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
    bal = (0.1 * rng.standard_normal(32)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=4, top_groups=2, group_top=2, scale=1.5)
    spec = q4.RouterSpec(balance=torch.from_numpy(bal).to(dev), **kw)
    r = q4.route_scored(layer, xd, spec)
    y = [q4.prefill(layer, xd, r)]
    if T <= q4.MAX_DECODE_TOKENS:
        ws = q4.workspace(layer, 1, dev)
        before = [t.clone() for t in (r.logits, r.topk_idx, r.topk_w)]
        y.append(q4.decode_tokens(layer, xd, ws, routing=r, routing_in=True))
        torch.cuda.synchronize()
        for a, b in zip(before, (r.logits, r.topk_idx, r.topk_w)):
            assert torch.equal(a, b)  # read, not written
    if T == 1:
        y.append(q4.decode(layer, xd, ws, routing=r, routing_in=True))
    torch.cuda.synchronize()
    logits = r.logits.cpu().numpy()
    ref = oracle.router_logits(x, L["w_router"], L["router_bias"])
    assert np.abs(logits - ref).max() <= 1e-3 * np.sqrt(np.mean(ref.astype(np.float64) ** 2))
    check(r, logits, 4, bal, **kw)
    idx, w = plain.route_scored(logits, 4, balance=bal, **kw)
    exact, _ = oracle.layer_tokens(L, x, np.arange(T), idx, w)
    rms = np.sqrt(np.mean(exact ** 2))
    bar = np.maximum(2e-2 * rms, np.abs(exact) * 2.0 ** -8 + 2e-3 * rms)
    for got in y:
        b = got.view(torch.int16).cpu().numpy().view(np.uint16)
        assert (np.abs(bits_to_f32(b) - exact) <= bar).all()


def test_decode_from_a_selection_equals_decode(dev):
    # moe_route's own selection handed to decode gives decode's own result, bit for bit
    rng = np.random.default_rng(4)
    L = random_layer(rng, 512, 128, 32, 4)
    layer = q4.DeviceLayer.from_host(L, dev)
    for T in (1, 5, 8):
        xd = torch.from_numpy(random_x(rng, T, 512).view(np.int16)).to(dev).view(torch.bfloat16)
        ws = q4.workspace(layer, 1, dev)
        r = q4.DeviceRouting(T, 32, 4, dev)
        want = q4.decode_tokens(layer, xd, ws, routing=r).clone()
        got = q4.decode_tokens(layer, xd, ws, routing=r, routing_in=True)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        # an index outside the experts is brought into range: the call stays in bounds
        r.topk_idx[0, 0] = 1 << 30
        r.topk_idx[T - 1, 1] = -5
        r.topk_idx[0, 2] = r.topk_idx[0, 3]  # and the same expert twice
        ref_idx = r.topk_idx.clamp(0, 31).clone()
        got = q4.decode_tokens(layer, xd, ws, routing=r, routing_in=True).clone()
        r.topk_idx.copy_(ref_idx)
        want = q4.decode_tokens(layer, xd, ws, routing=r, routing_in=True)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T", [7, 70])
def test_graph_replays(dev, T):
    E, k = 256, 8
    rng = np.random.default_rng(6)
    layer = small_layer(E, k, dev)
    kw = dict(score="sigmoid", n_groups=8, top_groups=4, group_top=2)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32)
    spec = q4.RouterSpec(balance=torch.from_numpy(b).to(dev), **kw)
    r = q4.DeviceRouting(T, E, k, dev)
    q4.route_scored(layer, None, spec, r, logits_in=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4.route_scored(layer, None, spec, r, logits_in=True)
    for rep in range(3):
        l = rng.standard_normal((T, E)).astype(np.float32)
        r.logits.copy_(torch.from_numpy(l))
        g.replay()
        torch.cuda.synchronize()
        check(r, l, k, b, **kw)
