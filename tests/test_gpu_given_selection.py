"""Decoding from a given selection through every entry point, and routing weights of
any size and sign through the experts' products.

Bars: the entry points run the same kernels, so bit-equal; against the oracle's layer
with the same selection that of the layer's own parity tests (2e-2 RMS, or half a bf16
step + 2e-3 RMS for large values)."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
import q4_routed_expert_amd as q4
from q4_routed_expert_amd import _abi
from workloads import bits_to_f32, random_layer, random_x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def case(dev, T, E=32, k=4, d=512, inter=128, seed=0):
    rng = np.random.default_rng(seed + T)
    L = random_layer(rng, d, inter, E, k, router_bias=True)
    x = random_x(rng, T, d)
    xd = torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
    return L, x, q4.DeviceLayer.from_host(L, dev), xd


@pytest.mark.parametrize("T", [1, 3, 8])
def test_static_scratch_takes_a_selection(dev, T):
    L, x, layer, xd = case(dev, T)
    spec = q4.RouterSpec(score="sigmoid", n_groups=4, top_groups=2, group_top=2, scale=2.5)
    r = q4.route_scored(layer, xd, spec)
    want = q4.decode_tokens(layer, xd, q4.workspace(layer, 1, dev), routing=r, routing_in=True)
    before = [t.clone() for t in (r.logits, r.topk_idx, r.topk_w)]
    y = torch.zeros_like(want)
    rc = _abi.lib().moe_decode_tokens_static(
        C.addressof(layer.struct), xd.data_ptr(), T, _abi.MOE_ROUTING_IN, C.addressof(r.struct),
        y.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, _abi.lib().moe_last_error().decode()
    torch.cuda.synchronize()
    assert np.array_equal(bits(y), bits(want))
    for a, b in zip(before, (r.logits, r.topk_idx, r.topk_w)):
        assert torch.equal(a, b)  # read, not written


@pytest.mark.parametrize("scale", [-0.5, 16.0, 300.0, 0.0])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_weights_of_any_size(dev, T, scale):
    # scaled weights, and slots of weight 0 and of opposite sign beside them
    L, x, layer, xd = case(dev, T, seed=40)
    r = q4.route_scored(layer, xd, q4.RouterSpec(score="sigmoid", renorm=False, scale=scale))
    r.topk_w[:, 1] *= -1.0
    r.topk_w[::2, 2] = 0.0
    y = [q4.prefill(layer, xd, r)]
    if T <= q4.MAX_DECODE_TOKENS:
        y.append(q4.decode_tokens(layer, xd, q4.workspace(layer, 1, dev), routing=r, routing_in=True))
    torch.cuda.synchronize()
    idx, w = r.topk_idx.cpu().numpy(), r.topk_w.cpu().numpy().astype(np.float64)
    tokens = np.arange(min(T, 40))
    exact, _ = oracle.layer_tokens(L, x, tokens, idx[tokens], w[tokens])
    rms = np.sqrt(np.mean(exact ** 2))
    bar = np.maximum(2e-2 * rms, np.abs(exact) * 2.0 ** -8 + 2e-3 * rms)
    for got in y:
        assert (np.abs(bits_to_f32(bits(got))[tokens] - exact) <= bar).all()


@pytest.mark.parametrize("E,k,inter", [(5, 1, 64), (130, 7, 192), (256, 8, 640)])
def test_other_layers(dev, E, k, inter):
    # no router work groups in the first kernel, whatever the shape
    for T in (1, 2, 4, 8):
        L, x, layer, xd = case(dev, T, E=E, k=k, d=448, inter=inter, seed=7)
        r = q4.DeviceRouting(T, E, k, dev)
        ws = q4.workspace(layer, 1, dev)
        want = q4.decode_tokens(layer, xd, ws, routing=r).clone()
        got = q4.decode_tokens(layer, xd, ws, routing=r, routing_in=True)
        torch.cuda.synchronize()
        assert np.array_equal(bits(got), bits(want)), T
