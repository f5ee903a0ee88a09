"""Refusals of the operators around the layer (scored routing, 4-bit products,
sampling, residual + norm), by the C ABI and by the binding.  No call here
reaches a kernel, so none needs a GPU."""
import ctypes as C

import pytest
import torch

import q4_routed_expert_amd as q4
from q4_routed_expert_amd import _abi

FAKE = 0x10000  # nonzero and aligned: validation only looks at addresses
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32


def _norm(**kw):
    a = dict(x=FAKE, T=4, d=128, residual=None, residual_out=None, weight=FAKE, eps=1e-6, flags=0,
             y=FAKE, y8=None, scale=None)
    a.update(kw)
    return _abi.lib().moe_add_norm(a["x"], a["T"], a["d"], a["residual"], a["residual_out"],
                                   a["weight"], a["eps"], a["flags"], a["y"], a["y8"], a["scale"],
                                   None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), _abi.MOE_EINVAL), (dict(T=_abi.MOE_MAX_TOKENS + 1), _abi.MOE_EUNSUPPORTED),
    (dict(d=0), _abi.MOE_EINVAL), (dict(d=100), _abi.MOE_EUNSUPPORTED),
    (dict(d=_abi.MOE_MAX_D + 64), _abi.MOE_EUNSUPPORTED),
    (dict(x=None), _abi.MOE_EINVAL), (dict(x=FAKE + 2), _abi.MOE_EINVAL),
    (dict(weight=None), _abi.MOE_EINVAL), (dict(residual=FAKE + 8), _abi.MOE_EINVAL),
    (dict(residual_out=FAKE), _abi.MOE_EINVAL),        # nothing to add
    (dict(y=None), _abi.MOE_EINVAL),                   # no output at all
    (dict(y8=FAKE), _abi.MOE_EINVAL), (dict(scale=FAKE), _abi.MOE_EINVAL),
    (dict(eps=-1.0), _abi.MOE_EINVAL), (dict(eps=float("nan")), _abi.MOE_EINVAL),
    (dict(eps=float("inf")), _abi.MOE_EINVAL), (dict(flags=4), _abi.MOE_EINVAL),
])
def test_add_norm_refuses(kw, code):
    assert _norm(**kw) == code
    assert _abi.lib().moe_last_error()


def test_add_norm_binding_refuses():
    x, w = torch.zeros(3, 128, dtype=bf16), torch.zeros(128, dtype=bf16)
    for kw, what in ((dict(x=x.float()), "x"), (dict(x=x[:, ::2]), "x"), (dict(x=x[0]), "x"),
                     (dict(weight=w[:64]), "weight"), (dict(weight=w.float()), "weight"),
                     (dict(residual=x.half()), "residual"), (dict(residual=x[:2]), "residual"),
                     (dict(residual=x, residual_out=x.float()), "residual_out"),
                     (dict(y=x.float()), "y"), (dict(y8=x), "y8"),
                     (dict(y8_scale=torch.zeros(5)), "y8_scale"), (dict(), "GPU")):
        a = dict(x=x, weight=w)
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.add_norm(a.pop("x"), a.pop("weight"), **a)
