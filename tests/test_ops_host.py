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
    (dict(residual=FAKE, residual_out=FAKE + 64, y=FAKE + 64), _abi.MOE_EINVAL),  # shared outputs
    (dict(y8=FAKE + 64, scale=FAKE, y=FAKE + 64), _abi.MOE_EINVAL),
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


def _spec(**kw):
    a = dict(score=0, n_groups=1, top_groups=1, group_top=1, renorm=1, scale=1.0, balance=None)
    a.update(kw)
    return _abi.RouterSpec(*[a[n] for n, _ in _abi.RouterSpec._fields_])


def _layer(E=256, k=8, d=128, inter=64, w_router=FAKE):
    return _abi.Layer(d, inter, E, k, w_router, None, *[_abi.Q4Mat() for _ in range(6)])


def _route(spec, layer=None, T=4, x=FAKE, flags=0, missing=None):
    L = layer or _layer()
    r = _abi.Routing(*[FAKE] * len(_abi.Routing._fields_))
    if missing:
        setattr(r, missing, None)
    return _abi.lib().moe_route_scored(C.addressof(L), x, T, flags,
                                       None if spec is None else C.addressof(spec),
                                       C.addressof(r), None)


@pytest.mark.parametrize("kw,code", [
    (dict(score=2), _abi.MOE_EINVAL), (dict(renorm=2), _abi.MOE_EINVAL),
    (dict(scale=float("nan")), _abi.MOE_EINVAL), (dict(scale=float("inf")), _abi.MOE_EINVAL),
    (dict(balance=FAKE + 4), _abi.MOE_EINVAL), (dict(n_groups=0), _abi.MOE_EINVAL),
    (dict(n_groups=8, top_groups=0), _abi.MOE_EINVAL),
    (dict(n_groups=8, top_groups=9), _abi.MOE_EINVAL),
    (dict(n_groups=128, top_groups=128), _abi.MOE_EUNSUPPORTED),
    (dict(n_groups=7, top_groups=7), _abi.MOE_EUNSUPPORTED),        # does not divide 256
    (dict(n_groups=8, top_groups=4, group_top=3), _abi.MOE_EUNSUPPORTED),
    (dict(n_groups=64, top_groups=1), _abi.MOE_EUNSUPPORTED),       # 4 experts, top-8
])
def test_route_scored_refuses_specs(kw, code):
    assert _route(_spec(**kw)) == code
    assert _abi.lib().moe_last_error()


def test_route_scored_refuses_arguments():
    s = _spec()
    assert _route(None) == _abi.MOE_EINVAL
    assert _route(s, T=0) == _abi.MOE_EINVAL
    assert _route(s, T=_abi.MOE_MAX_TOKENS + 1) == _abi.MOE_EUNSUPPORTED
    assert _route(s, flags=2) == _abi.MOE_EINVAL
    assert _route(s, flags=_abi.MOE_ROUTING_IN) == _abi.MOE_EINVAL
    assert _route(s, x=None) == _abi.MOE_EINVAL
    assert _route(s, layer=_layer(w_router=None)) == _abi.MOE_EINVAL
    assert _route(s, layer=_layer(E=257)) == _abi.MOE_EUNSUPPORTED
    assert _route(s, missing="blk_counts") == _abi.MOE_EINVAL


def test_decode_refuses_a_missing_selection():
    lib = _abi.lib()
    m = _abi.Q4Mat(FAKE, FAKE, FAKE)
    L = _abi.Layer(128, 64, 8, 2, FAKE, None, *[m] * 6)
    r = _abi.Routing(*[FAKE] * len(_abi.Routing._fields_))
    call = lambda flags, rr: lib.moe_decode_tokens(  # noqa: E731
        C.addressof(L), FAKE, 2, flags, rr, FAKE, 1 << 30, FAKE, None)
    assert call(_abi.MOE_ROUTING_IN, None) == _abi.MOE_EINVAL
    assert call(_abi.MOE_ROUTING_IN | _abi.MOE_LOGITS_IN, C.addressof(r)) == _abi.MOE_EINVAL
    r.topk_w = None
    assert call(_abi.MOE_ROUTING_IN, C.addressof(r)) == _abi.MOE_EINVAL
    assert b"topk_w" in lib.moe_last_error()


def test_route_scored_binding_refuses():
    import types
    L = types.SimpleNamespace(d=128, n_experts=8, top_k=2, inter=64, struct=None)
    with pytest.raises(ValueError, match="score"):
        q4.RouterSpec(score="tanh")
    with pytest.raises(ValueError, match="balance"):
        q4.RouterSpec(balance=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="logits_in"):
        q4.route_scored(L, None, q4.RouterSpec(), logits_in=True)
    r = q4.DeviceRouting(4, 8, 3, "cpu")
    with pytest.raises(ValueError, match="routing is for"):
        q4.route_scored(L, None, q4.RouterSpec(), r, logits_in=True)
    r = q4.DeviceRouting(4, 8, 2, "cpu")
    with pytest.raises(ValueError, match="routing is for"):
        q4.route_scored(L, torch.zeros(5, 128, dtype=bf16), q4.RouterSpec(), r)
    with pytest.raises(ValueError, match="balance"):
        q4.route_scored(L, None, q4.RouterSpec(balance=torch.zeros(7)), r, logits_in=True)
    with pytest.raises(ValueError, match="GPU"):
        q4.route_scored(L, None, q4.RouterSpec(), r, logits_in=True)
    ws = torch.empty(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="routing_in"):
        q4.decode_tokens(L, torch.zeros(2, 128, dtype=bf16), ws, routing_in=True)


def _linear(**kw):
    a = dict(q=FAKE, s=FAKE, b=FAKE, N=100, K=128, x=FAKE, T=4, flags=0, y=FAKE)
    a.update(kw)
    m = _abi.Q4Mat(a["q"], a["s"], a["b"])
    return _abi.lib().moe_linear(C.addressof(m), a["N"], a["K"], a["x"], a["T"], a["flags"], a["y"],
                                 None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), _abi.MOE_EINVAL), (dict(K=0), _abi.MOE_EINVAL), (dict(T=0), _abi.MOE_EINVAL),
    (dict(K=100), _abi.MOE_EUNSUPPORTED), (dict(K=_abi.MOE_MAX_D + 64), _abi.MOE_EUNSUPPORTED),
    (dict(N=_abi.MOE_MAX_VOCAB + 1), _abi.MOE_EUNSUPPORTED),
    (dict(T=_abi.MOE_MAX_LINEAR_TOKENS + 1), _abi.MOE_EUNSUPPORTED),
    (dict(flags=2), _abi.MOE_EINVAL), (dict(q=None), _abi.MOE_EINVAL),
    (dict(s=FAKE + 2), _abi.MOE_EINVAL), (dict(b=None), _abi.MOE_EINVAL),
    (dict(x=FAKE + 8), _abi.MOE_EINVAL), (dict(y=None), _abi.MOE_EINVAL),
    (dict(y=FAKE + 4), _abi.MOE_EINVAL),
])
def test_linear_refuses(kw, code):
    assert _linear(**kw) == code
    assert _abi.lib().moe_last_error()


def test_linear_binding_refuses():
    q = torch.zeros(10, 16, dtype=i32)
    s, x = torch.zeros(10, 2, dtype=bf16), torch.zeros(3, 128, dtype=bf16)
    for kw, what in ((dict(x=x[0]), "x must be"), (dict(x=x[:, :64]), "columns"),
                     (dict(x=x.float()), "x"), (dict(q=q.long()), "q"),
                     (dict(scale=s[:5]), "scale"), (dict(bias=s.float()), "bias"),
                     (dict(out_dtype=torch.float16), "out_dtype"),
                     (dict(y=torch.zeros(29)), "y"), (dict(q=q.t().contiguous().t()), "q"),
                     (dict(), "GPU")):
        a = dict(q=q, scale=s, bias=s, x=x)
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.linear(a.pop("q"), a.pop("scale"), a.pop("bias"), a.pop("x"), **a)


def _sample(V=100, B=4, d=0, logits=FAKE, token=FAKE, prob=None, x_next=None, ws=FAKE,
            ws_bytes=1 << 30, embed=None, **kw):
    lm = _abi.LmHead(V, d, _abi.Q4Mat(), embed or _abi.Q4Mat())
    p = _abi.Sampling(u=kw.pop("u", FAKE), **kw)
    return _abi.lib().moe_sample(C.addressof(lm), logits, B, C.addressof(p), token, prob, x_next, ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(V=0), _abi.MOE_EINVAL), (dict(B=0), _abi.MOE_EINVAL),
    (dict(V=_abi.MOE_MAX_VOCAB + 1), _abi.MOE_EUNSUPPORTED),
    (dict(B=_abi.MOE_MAX_SAMPLE_ROWS + 1), _abi.MOE_EUNSUPPORTED),
    (dict(logits=None), _abi.MOE_EINVAL), (dict(logits=FAKE + 4), _abi.MOE_EINVAL),
    (dict(u=None), _abi.MOE_EINVAL), (dict(u=FAKE + 2), _abi.MOE_EINVAL),
    (dict(temperature=FAKE + 1), _abi.MOE_EINVAL), (dict(top_k=FAKE + 2), _abi.MOE_EINVAL),
    (dict(top_p=FAKE + 2), _abi.MOE_EINVAL), (dict(min_p=FAKE + 3), _abi.MOE_EINVAL),
    (dict(token=None), _abi.MOE_EINVAL), (dict(token=FAKE + 2), _abi.MOE_EINVAL),
    (dict(prob=FAKE + 2), _abi.MOE_EINVAL), (dict(ws=None), _abi.MOE_EINVAL),
    (dict(ws_bytes=1000), _abi.MOE_EWORKSPACE),
    (dict(x_next=FAKE), _abi.MOE_EINVAL),                                    # d = 0
    (dict(x_next=FAKE, d=100), _abi.MOE_EUNSUPPORTED),
    (dict(x_next=FAKE, d=128), _abi.MOE_EINVAL),                             # no table
    (dict(x_next=FAKE + 8, d=128, embed=_abi.Q4Mat(FAKE, FAKE, FAKE)), _abi.MOE_EINVAL),
    # 4-byte aligned arrays are enough: these get as far as the workspace
    (dict(u=FAKE + 4, token=FAKE + 4, prob=FAKE + 12, top_k=FAKE + 8, ws_bytes=0),
     _abi.MOE_EWORKSPACE),
])
def test_sample_refuses(kw, code):
    assert _sample(**kw) == code
    assert _abi.lib().moe_last_error()


def test_sample_workspace_bytes():
    lib = _abi.lib()
    for V, B in ((1, 1), (248320, 64), (_abi.MOE_MAX_VOCAB, _abi.MOE_MAX_SAMPLE_ROWS)):
        assert lib.moe_sample_workspace_bytes(V, B) > 0
    for V, B in ((0, 1), (1, 0), (_abi.MOE_MAX_VOCAB + 1, 1), (10, _abi.MOE_MAX_SAMPLE_ROWS + 1)):
        assert lib.moe_sample_workspace_bytes(V, B) == 0
    for V in (1, 8192, 8193, 20000, 100003, 248320, _abi.MOE_MAX_VOCAB):  # more rows, more bytes
        sizes = [lib.moe_sample_workspace_bytes(V, B) for B in range(1, 200)]
        assert all(a < b for a, b in zip(sizes, sizes[1:])), V


def test_sample_binding_refuses():
    import types
    l, u = torch.zeros(3, 50), torch.zeros(3)
    lm = types.SimpleNamespace(V=50, d=128, embed={}, struct=None)
    for kw, what in ((dict(logits=l[0]), "logits"), (dict(logits=l.double()), "logits"),
                     (dict(logits=l.t()), "logits"), (dict(u=u[:2]), "u"), (dict(u=u.double()), "u"),
                     (dict(temperature=u[:1]), "temperature"), (dict(top_k=u), "top_k"),
                     (dict(top_p=u.half()), "top_p"), (dict(min_p=u.int()), "min_p"),
                     (dict(token=u), "token"), (dict(prob=u.double()), "prob"),
                     (dict(x_next=torch.zeros(3, 128, dtype=bf16)), "x_next"),
                     (dict(x_next=torch.zeros(2, 128, dtype=bf16), lm=lm), "x_next"),
                     (dict(top_k=2**32 + 1), "top_k"), (dict(ws=u), "ws"),
                     (dict(ws=torch.empty(10, dtype=torch.uint8)), "GPU")):
        a = dict(logits=l, u=u)
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.sample(a.pop("logits"), a.pop("u"), **a)


def test_every_finite_number_is_taken():
    # the largest fp32 numbers get as far as the next check
    big = torch.finfo(f32).max
    for scale in (big, -big):
        assert _route(_spec(scale=scale, n_groups=0)) == _abi.MOE_EINVAL
        assert b"n_groups" in _abi.lib().moe_last_error()
    assert _norm(eps=big, x=None) == _abi.MOE_EINVAL
    assert b"x is NULL" in _abi.lib().moe_last_error()

