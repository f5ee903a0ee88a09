"""Calls on a stream that is not the current one.

Each call below is given its inputs only and allocates everything else.  On the CPU:
every allocation happens with the call's stream current (a tensor from another
stream's pool may still be in use there, its zero fill is not ordered before the
kernels, and a dropped workspace goes to that stream's next tensor).  The calls are
refused afterwards, because the tensors are not on the GPU.  On the GPU: the results
are those of the current stream, while the current stream allocates and fills memory
of the same sizes right after each call."""
import contextlib
import types

import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import q4_routed_expert_amd as q4
from workloads import random_layer, random_lm, random_x

bf16 = torch.bfloat16


class Allocations(TorchDispatchMode):
    """(operation, was the call's stream current) of every allocation."""

    def __init__(self):
        super().__init__()
        self.seen, self.active = [], False

    def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
        name = func.overloadpacket.__name__
        if "empty" in name or "zeros" in name:
            self.seen.append((name, self.active))
        return func(*args, **(kwargs or {}))


def _calls(layer, lm, dev):
    x = torch.ones(4, 128, dtype=bf16, device=dev)
    l, u = torch.zeros(4, 50, device=dev), torch.zeros(4, device=dev)
    w = torch.ones(128, dtype=bf16, device=dev)
    q = torch.zeros(10, 16, dtype=torch.int32, device=dev)
    sc = torch.zeros(10, 2, dtype=bf16, device=dev)
    ws = torch.zeros(16, dtype=torch.uint8, device=dev)
    r = q4.DeviceRouting(4, 8, 2, dev)
    return {
        "route": (lambda s: q4.route(layer, x, stream=s), 12),
        "route_scored": (lambda s: q4.route_scored(layer, x, q4.RouterSpec(), stream=s), 12),
        "prefill": (lambda s: q4.prefill(layer, x, r, stream=s), 2),
        "decode": (lambda s: q4.decode(layer, x[:1], ws, stream=s), 1),
        "decode_tokens": (lambda s: q4.decode_tokens(layer, x, ws, stream=s), 1),
        "lm_argmax": (lambda s: q4.lm_argmax(lm, x[0], ws, stream=s), 2),
        "linear": (lambda s: q4.linear(q, sc, sc, x, stream=s), 1),
        "sample": (lambda s: q4.sample(l, u, stream=s), 3),
        "add_norm": (lambda s: q4.add_norm(x, w, stream=s), 1),
        "add_norm_e4m3": (lambda s: q4.add_norm(x, w, e4m3=True, stream=s), 2),
    }


NAMES = ("route", "route_scored", "prefill", "decode", "decode_tokens", "lm_argmax", "linear",
         "sample", "add_norm", "add_norm_e4m3")


@pytest.mark.parametrize("name", NAMES)
def test_own_buffers_come_from_the_calls_stream(name, monkeypatch):
    L = random_layer(np.random.default_rng(0), 128, 64, 8, 2)
    layer = q4.DeviceLayer.from_host(L, "cpu")
    lm = types.SimpleNamespace(V=50, d=128, struct=None)
    call, n = _calls(layer, lm, "cpu")[name]
    mode = Allocations()
    stream = types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0)

    @contextlib.contextmanager
    def current(s):
        assert s is stream
        mode.active = True
        yield
        mode.active = False

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    with mode, pytest.raises(ValueError, match="GPU"):
        call(stream)
    assert len(mode.seen) >= n and all(active for _, active in mode.seen), mode.seen


@pytest.mark.gpu
def test_results_on_another_stream():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(1)
    layer = q4.DeviceLayer.from_host(random_layer(rng, 512, 128, 32, 4), dev)
    _, head, embed = random_lm(rng, 20000, 512)
    lm = q4.DeviceLmHead.from_host(head, embed, dev)
    x = torch.from_numpy(random_x(rng, 600, 512).view(np.int16)).to(dev).view(bf16)
    l, u = 2 * torch.randn(8, 20000, device=dev), torch.rand(8, device=dev)
    w = torch.ones(512, dtype=bf16, device=dev)
    ws, lws = q4.workspace(layer, 1, dev), q4.lm_workspace(lm, dev)
    # (the tail of block_map and of the other maps is not written: zeros in both)
    arrays = lambda r: [getattr(r, f) for f, _ in q4._abi.Routing._fields_]         # noqa: E731
    given = q4.route(layer, x)
    calls = [
        lambda s: arrays(q4.route(layer, x, stream=s)),
        lambda s: arrays(q4.route_scored(layer, x, q4.RouterSpec(), stream=s)),
        lambda s: arrays(q4.route_scored(layer, x[:9], q4.RouterSpec(), stream=s)),
        lambda s: [q4.prefill(layer, x, given, stream=s)],
        lambda s: [q4.decode(layer, x[:1], ws, stream=s)],
        lambda s: [q4.decode_tokens(layer, x[:5], ws, stream=s)],
        lambda s: list(q4.lm_argmax(lm, x[0], lws, stream=s)[:2]),
        lambda s: [q4.linear(head_q, head_s, head_b, x[:7], stream=s)],
        lambda s: list(q4.sample(l, u, top_k=100, top_p=0.9, stream=s)[:2]),
        lambda s: list(q4.add_norm(x, w, e4m3=True, stream=s)[1:]),
    ]
    head_q, head_s, head_b = (lm.head[n] for n in ("q", "scale", "bias"))
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        for _ in range(3):
            got = call(side)
            # memory of the sizes a dropped workspace or an unordered fill would share
            junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
                    for n in (1 << 10, 1 << 16, 1 << 20, 1 << 23)]
            torch.cuda.current_stream().wait_stream(side)
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
            del got, junk


@pytest.mark.gpu
def test_captured_on_a_forked_stream():
    # the workspace of sample is allocated and dropped inside the capture
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    l, u = 2 * torch.randn(5, 30000, device=dev), torch.rand(5, device=dev)
    x, w = torch.randn(5, 512, device=dev).to(bf16), torch.ones(512, dtype=bf16, device=dev)
    side = torch.cuda.Stream()
    q4.sample(l, u, top_p=0.9)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        a = q4.sample(l, u, top_p=0.9, stream=side)
        b = q4.sample(l, u, top_k=40, stream=side)
        c = q4.add_norm(x, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for rep in range(3):
        l.copy_(2 * torch.randn(5, 30000, device=dev))
        u.uniform_()
        x.copy_(torch.randn(5, 512, device=dev))
        g.replay()
        torch.cuda.synchronize()
        for got, want in ((a, q4.sample(l, u, top_p=0.9)), (b, q4.sample(l, u, top_k=40)),
                          (c, q4.add_norm(x, w))):
            for s, t in zip(got, want):
                assert (s is None and t is None) or torch.equal(s, t), rep
