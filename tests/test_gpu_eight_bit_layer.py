"""The 8-bit operators together, as a layer of a model with e4m3 experts and the step from its
head to a token run them: residual + norm (bf16 and e4m3 rows at once), scored routing, rows
into expert order, gate/up and down products by expert, the shared expert's products on the
norm's e4m3 rows, rows back to their tokens on top of it, the 4-bit head, penalties with a
grammar's mask, sampling.

Each stage is checked against its definition on the values the stage before it left on the
GPU, with the bars of the operators' own tests; then captured steps against eager ones, and two
streams at once, bit for bit; then the way back through the expert rows."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain
from routings import values
from test_gpu_scaled_products import CUT, bar_of, check, check_gated, gated
from workloads import random_lm

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16
D, INTER, E, K, V = 448, 192, 24, 4, 9001
SAMPLE = dict(temperature=0.9, top_k=100, top_p=0.95)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def wide(t):
    return t.float().cpu().numpy().astype(np.float64)


class Step:
    def __init__(self, dev, T):
        rng = np.random.default_rng(70 + T)
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))   # noqa: E731
        q = lambda *s: tuple(t.to(dev) for t in q4.quantize_blocks(f(*s) * s[-1] ** -0.5))  # noqa: E731
        self.T = T
        self.x, self.res = f(T, D).to(dev).to(bf16), f(T, D).to(dev).to(bf16)
        self.nw = (1 + 0.1 * f(D)).to(dev).to(bf16)
        t = {m + "_q": torch.zeros(E * 64 * 8, dtype=torch.int32, device=dev) for m in q4.MATS}
        t |= {m + z: torch.zeros(E * 64, dtype=torch.int16, device=dev) for m in q4.MATS
              for z in ("_s", "_b")}
        t["w_router"] = (f(D, E) * D ** -0.5).to(dev)
        self.layer = q4.DeviceLayer(D, 64, E, K, t)
        self.spec = q4.RouterSpec(score="sigmoid", scale=1.5)
        self.w13, self.s13 = q(E, 2, INTER, D)
        self.w2, self.s2 = q(E, D, INTER)
        self.sh13, self.shs13 = q(2, INTER, D)
        self.sh2, self.shs2 = q(D, INTER)
        _, self.head, _ = random_lm(rng, V, D)
        self.lm = q4.DeviceLmHead.from_host(self.head, None, dev)
        self.r = q4.DeviceRouting(T, E, K, dev)
        self.n = torch.zeros(T, D, dtype=bf16, device=dev)
        self.history = torch.from_numpy(rng.integers(-1, 60, (T, 40)).astype(np.int32)).to(dev)
        allowed = rng.random((T, V)) < 0.5
        self.allowed = allowed
        bits = np.zeros((T, -(-V // 32) * 32), np.uint8)
        bits[:, :V] = allowed
        self.mask = torch.from_numpy(np.packbits(bits, 1, bitorder="little").view(np.int32).copy()).to(dev)
        self.u = torch.full((T,), 0.4, device=dev)
        self.ws = q4.sample_workspace(T, V, dev)

    def run(self):
        T = self.T
        _, self.n8, self.ns = q4.add_norm(self.x, self.nw, self.res, y=self.n, e4m3=True, group=128)
        q4.route_scored(self.layer, self.n, self.spec, self.r)
        self.rows, self.rs = q4.dispatch(self.n, self.r, e4m3=True)
        self.h, self.hs = q4.experts_e4m3(self.w13, self.s13, self.rows, self.rs, self.r, gated=True)
        self.e = q4.experts_e4m3(self.w2, self.s2, self.h, self.hs, self.r)
        self.sh, self.shs = q4.linear_e4m3(self.sh13, self.shs13, self.n8, self.ns, gated=True)
        self.base = q4.linear_e4m3(self.sh2, self.shs2, self.sh, self.shs)
        self.y = q4.combine(self.e, self.r, base=self.base)
        m = min(T, q4.MAX_LINEAR_TOKENS)
        hd = self.lm.head
        self.logits = q4.linear(hd["q"], hd["scale"], hd["bias"], self.y[:m])
        self.pen = q4.penalize(self.logits, tokens=self.history[:m], repetition=1.2, frequency=0.1,
                               presence=0.2, mask=self.mask[:m])
        self.token, self.prob, _ = q4.sample(self.pen, self.u[:m], ws=self.ws, **SAMPLE)
        return [self.n, self.n8, self.ns, self.rows, self.rs, self.h, self.hs, self.e, self.sh, self.shs,
                self.base, self.y, self.logits, self.pen, self.token, self.prob]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 7, 64, 600])
def test_a_step_follows_the_definitions(dev, T):
    s = Step(dev, T)
    s.run()
    torch.cuda.synchronize()
    v = wide((s.x.float() + s.res.float()).to(bf16))
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * wide(s.nw)
    assert (np.abs(wide(s.n) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -17)).all()
    sc = plain.expand(wide(s.ns), 1, T, D)
    bar = np.maximum(np.abs(want) * 2.0 ** -4, sc * 2.0 ** -10) + np.abs(want) * 2.0 ** -16
    assert (np.abs(values(s.n8) * sc - want) <= bar).all()
    idx, w = plain.route_scored(s.r.logits.cpu().numpy(), K, score="sigmoid", scale=1.5)
    assert np.array_equal(s.r.topk_idx.cpu().numpy(), idx)
    o = plain.sort_assignments(idx, E)
    n = wide(s.n)[o["perm"] // K]
    sc = plain.expand(wide(s.rs), 1, T * K, D)
    bar = np.maximum(np.abs(n) * 2.0 ** -4, sc * 2.0 ** -10) + np.abs(n) * 2.0 ** -20
    assert (np.abs(values(s.rows) * sc - n) <= bar).all()
    for e in range(E):
        a, b = int(o["offsets"][e]), int(o["offsets"][e + 1])
        if a == b:
            continue
        h, eh = gated(s.w13[e].cpu(), s.s13[e].cpu(), s.rows[a:b].cpu(), s.rs[a:b].cpu())
        check_gated(s.h[a:b], s.hs[a:b], h, eh)
        y, size = plain.product(values(s.w2[e]), wide(s.s2[e]), values(s.h[a:b]), wide(s.hs[a:b]))
        check(s.e[a:b], y, bar_of(size, INTER) + np.abs(y) * 2.0 ** -8 + CUT * size)
    h, eh = gated(s.sh13.cpu(), s.shs13.cpu(), s.n8.cpu(), s.ns.cpu())
    check_gated(s.sh, s.shs, h, eh)
    y, size = plain.product(values(s.sh2), wide(s.shs2), values(s.sh), wide(s.shs))
    check(s.base, y, bar_of(size, INTER) + np.abs(y) * 2.0 ** -8 + CUT * size)
    inv, wt = o["inv_perm"].reshape(T, K), wide(s.r.topk_w)
    assert (np.abs(wt - w) <= 2.0 ** -20 * np.abs(w)).all()
    y = plain.combine(wide(s.e), inv, wt, wide(s.base))
    size = plain.combine(np.abs(wide(s.e)), inv, np.abs(wt), np.abs(wide(s.base)))
    check(s.y, y, (K + 1) * 2.0 ** -24 * size + np.abs(y) * 2.0 ** -8)
    logits, pen = s.logits.cpu().numpy(), s.pen.cpu().numpy()
    for b in range(min(T, 9)):
        p, size = plain.penalize(logits[b], s.history[b].cpu().numpy(), 0, 1.2, 0.1, 0.2,
                                 allowed=s.allowed[b])
        assert np.array_equal(np.isinf(pen[b]), ~s.allowed[b])
        ok = s.allowed[b]
        assert (np.abs(pen[b][ok] - p[ok]) <= 4 * 2.0 ** -24 * size[ok]).all()
        tok, prob = plain.sample(pen[b], 0.4, **SAMPLE)
        assert int(s.token[b]) == tok and s.allowed[b][tok]
        assert abs(float(s.prob[b]) - prob) <= prob * 2.0 ** -24 + 2.0 ** -30


@pytest.mark.parametrize("T", [3, 300])
def test_captured_steps_match_eager_ones(dev, T):
    s = Step(dev, T)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.run()
    for i in range(3):
        s.x.copy_(torch.randn(T, D, device=dev))
        s.u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        torch.zeros(16, device=dev).sum()  # eager work between replays
        assert same(got, s.run()), i


def test_two_graphs_and_two_streams_at_once(dev):
    steps = [Step(dev, 5), Step(dev, 90)]
    want = [[t.clone() for t in s.run()] for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        outs = []
        for st, s in zip(streams, steps):
            with torch.cuda.stream(st):
                outs.append(s.run())
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.run()
        graphs.append((g, out))
    for _ in range(3):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(out, b) for (_, out), b in zip(graphs, want))


def test_the_way_back(dev):
    # the gradients of combine and dispatch around a linear map of the expert rows, against
    # the formula: y = sum_s w (2 rows(x)) gives dx = 2 (sum_s w) dy
    T = 33
    s = Step(dev, T)
    s.run()
    rows, _ = q4.dispatch(s.n, s.r)
    dy = torch.randn(T, D, device=dev).to(bf16)
    d_rows, d_w = q4.combine_grad(dy, 2 * rows, s.r)
    dx = q4.combine(2 * d_rows, s.r, weighted=False)
    w = wide(s.r.topk_w)
    want = 2 * w.sum(1, keepdims=True) * wide(dy)
    # K gradients and their sum, each rounded to bf16
    bar = 2 * np.abs(w).sum(1, keepdims=True) * np.abs(wide(dy)) * (2.0 ** -7 + 2.0 ** -20)
    assert (np.abs(wide(dx) - want) <= bar).all()
    dot = 2 * (wide(s.n) * wide(dy)).sum(1)
    size = 2 * np.abs(wide(s.n) * wide(dy)).sum(1)
    assert (np.abs(wide(d_w) - dot[:, None]) <= 50 * 2.0 ** -24 * size[:, None]).all()


def test_own_buffers_come_from_the_calls_stream(dev):
    s = Step(dev, 200)
    calls = [lambda st: q4.dispatch(s.n, s.r, e4m3=True, stream=st),
             lambda st: q4.experts_e4m3(s.w13, s.s13, s.rows, s.rs, s.r, gated=True, stream=st),
             lambda st: (q4.experts_e4m3(s.w2, s.s2, s.h, s.hs, s.r, stream=st),),
             lambda st: q4.linear_e4m3(s.sh13, s.shs13, s.n8, s.ns, gated=True, stream=st),
             lambda st: (q4.combine(s.e, s.r, base=s.base, stream=st),),
             lambda st: q4.combine_grad(s.n, s.e, s.r, stream=st),
             lambda st: (q4.penalize(s.logits, tokens=s.history[:64], frequency=1.0, stream=st),)]
    s.run()
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        for _ in range(3):
            got = call(side)
            junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
                    for n in (1 << 10, 1 << 16, 1 << 20, 1 << 23)]
            torch.cuda.current_stream().wait_stream(side)
            assert same(got, want), i
            del got, junk
