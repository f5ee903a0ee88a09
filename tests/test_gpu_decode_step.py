"""The operators together, as a decode step of a few sequences runs them: residual +
norm, scored routing, the experts' decode products with that selection, residual +
norm, the 4-bit output head, sampling, and the sampled tokens' embedding rows as the
next step's input.

Each stage is checked against its definition on the values the stage before it left
on the GPU (so errors do not add up along the chain), with the bars of the
operators' own tests; then captured steps against eager ones, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import q4_routed_expert_amd as q4
from oracle import operators as plain
from workloads import bits_to_f32, random_layer, random_lm

pytestmark = pytest.mark.gpu

D, E, K, V = 512, 32, 4, 20000
ROUTE = dict(score="sigmoid", n_groups=4, top_groups=2, group_top=2, scale=1.5)
SAMPLE = dict(temperature=0.9, top_k=200, top_p=0.95, min_p=0.001)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Step:
    def __init__(self, dev, B):
        rng = np.random.default_rng(50 + B)
        self.B, self.L = B, random_layer(rng, D, 128, E, K)
        _, self.head, self.embed = random_lm(rng, V, D)
        self.layer = q4.DeviceLayer.from_host(self.L, dev)
        self.lm = q4.DeviceLmHead.from_host(self.head, self.embed, dev)
        self.balance = (0.1 * rng.standard_normal(E)).astype(np.float32)
        self.spec = q4.RouterSpec(balance=torch.from_numpy(self.balance).to(dev), **ROUTE)
        self.w1, self.w2 = (torch.from_numpy(1 + 0.1 * rng.standard_normal(D).astype(np.float32))
                            .to(dev).to(torch.bfloat16) for _ in range(2))
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)           # noqa: E731
        self.x, self.res, self.n1, self.y, self.n2 = (bf(B, D) for _ in range(5))
        self.x.copy_(torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)))
        self.routing = q4.DeviceRouting(B, E, K, dev)
        self.logits = torch.zeros(B, V, device=dev)
        self.u = torch.zeros(B, device=dev)
        self.token = torch.zeros(B, dtype=torch.int32, device=dev)
        self.prob = torch.zeros(B, device=dev)
        self.ws = q4.workspace(self.layer, 1, dev)
        self.sws = q4.sample_workspace(B, V, dev)

    def run(self):
        q4.add_norm(self.x, self.w1, self.res, residual_out=self.res, y=self.n1)
        q4.route_scored(self.layer, self.n1, self.spec, self.routing)
        q4.decode_tokens(self.layer, self.n1, self.ws, y=self.y, routing=self.routing,
                         routing_in=True)
        q4.add_norm(self.y, self.w2, self.res, residual_out=self.res, y=self.n2)
        h = self.lm.head
        q4.linear(h["q"], h["scale"], h["bias"], self.n2, y=self.logits)
        q4.sample(self.logits, self.u, lm=self.lm, token=self.token, prob=self.prob,
                  x_next=self.x, ws=self.sws, **SAMPLE)

    def state(self):
        return [t.clone() for t in (self.x, self.res, self.n1, self.y, self.n2, self.logits,
                                    self.token, self.prob)]


def norm(x, w):
    v = x.float().cpu().numpy().astype(np.float64)
    return v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * w.float().cpu().numpy()


@pytest.mark.parametrize("B", [1, 5, 8])
def test_a_step_follows_the_definitions(dev, B):
    s = Step(dev, B)
    for step in range(2):
        x0, r0 = s.x.clone(), s.res.clone()
        s.u.copy_(torch.linspace(0.1, 0.9, B))
        s.run()
        torch.cuda.synchronize()
        r1 = (x0.float() + r0.float()).to(torch.bfloat16)
        want = norm(r1, s.w1)
        n1 = s.n1.float().cpu().numpy().astype(np.float64)
        assert (np.abs(n1 - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -17)).all()
        lg = s.routing.logits.cpu().numpy()
        ref = oracle.router_logits(bits(s.n1), s.L["w_router"])
        assert np.abs(lg - ref).max() <= 1e-3 * np.sqrt(np.mean(ref.astype(np.float64) ** 2))
        idx, w = plain.route_scored(lg, K, balance=s.balance, **ROUTE)
        assert np.array_equal(s.routing.topk_idx.cpu().numpy(), idx)
        exact, _ = oracle.layer_tokens(s.L, bits(s.n1), np.arange(B), idx, w)
        rms = np.sqrt(np.mean(exact ** 2))
        bar = np.maximum(2e-2 * rms, np.abs(exact) * 2.0 ** -8 + 2e-3 * rms)
        assert (np.abs(bits_to_f32(bits(s.y)) - exact) <= bar).all()
        r2 = (r1.float() + s.y.float()).to(torch.bfloat16)
        assert torch.equal(s.res, r2)
        want = norm(r2, s.w2)
        n2 = s.n2.float().cpu().numpy().astype(np.float64)
        assert (np.abs(n2 - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -17)).all()
        logits = s.logits.cpu().numpy()
        want = plain.linear(s.head["q"], s.head["scale"], s.head["bias"], n2)
        bar = 8 * np.sqrt(D) * 2.0 ** -24 * 0.13 * np.abs(n2).sum(1)[:, None]
        assert (np.abs(logits - want) <= bar).all()
        u = s.u.cpu().numpy()
        for b in range(B):
            tok, p = plain.sample(logits[b], u[b], **SAMPLE)
            assert int(s.token[b]) == tok
            assert abs(float(s.prob[b]) - p) <= p * 2.0 ** -24 + 2.0 ** -30
            row = oracle.embed_row(s.embed["q"], s.embed["scale"], s.embed["bias"], tok)
            assert np.array_equal(bits(s.x[b]), row)


def test_captured_steps_match_eager_ones(dev):
    B = 6
    eager, captured = Step(dev, B), Step(dev, B)
    us = torch.rand(4, B, device=dev)
    want = []
    for i in range(4):
        eager.u.copy_(us[i])
        eager.run()
        want.append(eager.state())
    start = [captured.x.clone(), captured.res.clone()]
    captured.run()  # warm-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured.run()
    captured.x.copy_(start[0])
    captured.res.copy_(start[1])
    for i in range(4):
        captured.u.copy_(us[i])
        g.replay()
        torch.cuda.synchronize()
        _ = torch.zeros(16, device=dev).sum()  # eager work between replays
        for a, b in zip(captured.state(), want[i]):
            assert torch.equal(a, b), i


def test_two_steps_at_once_on_two_streams(dev):
    # each with buffers and workspaces of its own: they may overlap in any way
    steps = [Step(dev, 4), Step(dev, 7)]
    for s in steps:
        s.u.fill_(0.4)
    refs = []
    for s in steps:
        x, r = s.x.clone(), s.res.clone()
        s.run()
        torch.cuda.synchronize()
        refs.append(s.state())
        s.x.copy_(x)
        s.res.copy_(r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for st, s in zip(streams, steps):
        with torch.cuda.stream(st):
            s.run()
    torch.cuda.synchronize()
    for s, ref in zip(steps, refs):
        for a, b in zip(s.state(), ref):
            assert torch.equal(a, b)
