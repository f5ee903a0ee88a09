"""Refusals of the 8-bit products, the calls around expert order, penalize and add_norm's
groups of 128, by the C ABI and by the binding.  No call here reaches a kernel, so none
needs a GPU."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from q4_routed_expert_amd import _abi
from routings import device_routing, quantised_rows, selections, values

FAKE = 0x10000  # nonzero and aligned: validation only looks at addresses
OTHER = 0x20000
bf16, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
EINVAL, EUNSUPPORTED = _abi.MOE_EINVAL, _abi.MOE_EUNSUPPORTED


def routing(**kw):
    r = _abi.Routing(*[FAKE] * len(_abi.Routing._fields_))
    for n, v in kw.items():
        setattr(r, n, v)
    return r


def linear(**kw):
    a = dict(w=FAKE, ws=FAKE, N=256, K=128, x=FAKE, xs=FAKE + 64, T=4, flags=0, y=OTHER, y_scale=None)
    a.update(kw)
    m = _abi.E4m3Mat(a["w"], a["ws"])
    return _abi.lib().moe_linear_scaled(C.addressof(m), a["N"], a["K"], a["x"], a["xs"], a["T"],
                                        a["flags"], a["y"], a["y_scale"], None)


def experts(r=None, **kw):
    a = dict(E=8, N=256, K=128, T=4, k=2, flags=0, y=OTHER, y_scale=None, x=FAKE)
    a.update(kw)
    m = _abi.E4m3Mat(FAKE, FAKE)
    r = routing() if r is None else r
    return _abi.lib().moe_experts_scaled(C.addressof(m), a["E"], a["N"], a["K"], a["x"], FAKE, a["T"],
                                         a["k"], C.addressof(r) if r else None, a["flags"], a["y"],
                                         a["y_scale"], None)


PRODUCT = [(dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(K=100), EUNSUPPORTED),
           (dict(K=_abi.MOE_MAX_D + 64), EUNSUPPORTED), (dict(N=_abi.MOE_MAX_VOCAB + 1), EUNSUPPORTED),
           (dict(T=0), EINVAL), (dict(T=_abi.MOE_MAX_TOKENS + 1), EUNSUPPORTED),
           (dict(flags=4), EINVAL), (dict(flags=3, y_scale=OTHER + 64), EINVAL),
           (dict(flags=2), EINVAL), (dict(y_scale=OTHER + 64), EINVAL),
           (dict(flags=2, y_scale=OTHER + 64, N=192), EUNSUPPORTED),
           (dict(flags=2, y_scale=OTHER), EINVAL), (dict(x=None), EINVAL), (dict(x=FAKE + 8), EINVAL),
           (dict(y=None), EINVAL), (dict(y=FAKE), EINVAL)]


@pytest.mark.parametrize("call", [linear, experts])
@pytest.mark.parametrize("kw,code", PRODUCT)
def test_products_refuse(call, kw, code):
    assert call(**kw) == code
    assert _abi.lib().moe_last_error()


def test_products_refuse_more():
    assert linear(w=None) == linear(ws=None) == linear(xs=None) == linear(xs=FAKE + 4) == EINVAL
    assert _abi.lib().moe_linear_scaled(None, 256, 128, FAKE, FAKE, 1, 0, OTHER, None, None) == EINVAL
    assert experts(E=0) == experts(k=0) == EINVAL
    assert experts(E=257) == experts(k=9) == experts(E=3, k=4) == EUNSUPPORTED
    assert experts(r=False) == EINVAL
    for n in ("offsets", "block_map", "n_blocks", "tile_map", "n_tiles"):
        assert experts(r=routing(**{n: None})) == EINVAL


def test_expert_order_refuses():
    lib, r = _abi.lib(), routing()
    p = C.addressof(r)
    dispatch = lambda x=FAKE, T=4, k=2, d=128, r=p, rows=OTHER, s=None: lib.moe_dispatch(  # noqa: E731
        x, T, k, d, r, rows, s, None)
    combine = lambda x=FAKE, T=4, k=2, d=128, r=p, flags=0, base=None, y=OTHER: lib.moe_combine(  # noqa: E731
        x, T, k, d, r, flags, base, y, None)
    grad = lambda x=FAKE, T=4, k=2, d=128, r=p, rows=FAKE + 64, dr=OTHER, dw=OTHER + 64: (  # noqa: E731
        lib.moe_combine_grad(x, rows, T, k, d, r, dr, dw, None))
    none = routing(inv_perm=None)
    for call in (dispatch, combine, grad):
        assert call(T=0) == call(k=0) == call(d=0) == call(x=None) == call(r=None) == EINVAL
        assert call(r=C.addressof(none)) == call(x=FAKE + 2) == EINVAL
        assert call(T=_abi.MOE_MAX_TOKENS + 1) == call(k=9) == call(d=96) == EUNSUPPORTED
        assert call(d=_abi.MOE_MAX_D + 64) == EUNSUPPORTED
    assert dispatch(rows=None) == dispatch(rows=FAKE) == dispatch(s=OTHER) == dispatch(s=FAKE) == EINVAL
    assert combine(flags=2) == combine(y=FAKE) == combine(y=None) == combine(base=FAKE + 4) == EINVAL
    weightless = routing(topk_w=None)
    assert combine(r=C.addressof(weightless)) == grad(r=C.addressof(weightless)) == EINVAL
    assert grad(rows=None) == grad(dr=None) == grad(dw=None) == grad(dr=FAKE) == grad(dw=OTHER) == EINVAL


def penalties(**kw):
    p = _abi.Penalties()
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def penalize(p, logits=FAKE, B=2, V=100, out=OTHER):
    return _abi.lib().moe_penalize(logits, B, V, C.addressof(p) if p else None, out, None)


def test_penalize_refuses():
    ok = penalties()
    assert penalize(None) == EINVAL
    assert penalize(ok, logits=None) == penalize(ok, out=None) == penalize(ok, logits=FAKE + 4) == EINVAL
    assert penalize(ok, B=0) == penalize(ok, V=0) == EINVAL
    assert penalize(ok, B=_abi.MOE_MAX_SAMPLE_ROWS + 1) == EUNSUPPORTED
    assert penalize(ok, V=_abi.MOE_MAX_VOCAB + 1) == EUNSUPPORTED
    for bad in (dict(tokens=FAKE + 2), dict(tokens=FAKE, stride=-1), dict(n_tokens=FAKE),
                dict(n_prompt=FAKE), dict(bias_ids=FAKE), dict(bias=FAKE),
                dict(bias_ids=FAKE, bias=FAKE, n_bias=-1), dict(mask=FAKE + 1),
                dict(repetition=FAKE + 2)):
        assert penalize(penalties(**bad)) == EINVAL, bad
    assert penalize(penalties(bias_ids=FAKE, bias=FAKE, n_bias=1025)) == EUNSUPPORTED
    assert penalize(penalties(tokens=FAKE, stride=_abi.MOE_MAX_HISTORY + 1)) == EUNSUPPORTED


def test_struct_sizes_and_limits_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "q4moe.h")).read()
    for name in ("MOE_E4M3_BLOCK", "MOE_MAX_BIASES", "MOE_MAX_HISTORY", "MOE_GATED", "MOE_UNWEIGHTED",
                 "MOE_NORM_GROUP_128"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(_abi, name), name
    assert C.sizeof(_abi.Penalties) == 9 * 8 + 5 * 4 + 4 and C.sizeof(_abi.E4m3Mat) == 16
    v = (*range(1, 10), 10, 11, 1.5, 2.5, 3.5)
    assert bytes(_abi.Penalties(*v)) == _abi.PENALTIES(*v)


def test_product_binding_refuses():
    x, xs = torch.zeros(4, 192).to(f8), torch.zeros(4, 2)
    w, ws = torch.zeros(130, 192).to(f8), torch.zeros(2, 2)
    for kw, what in ((dict(x=x.float()), "x"), (dict(x=x[0]), "x"), (dict(x=x[:, :128]), "columns"),
                     (dict(w=w.float()), "w"), (dict(w=w[None]), "w"), (dict(ws=ws[:1]), "w_scale"),
                     (dict(ws=ws.half()), "w_scale"), (dict(xs=xs[:3]), "x_scale"),
                     (dict(xs=torch.zeros(4, 3)), "x_scale"),  # a scale per 64 columns
                     (dict(ws=torch.zeros(3, 2)), "w_scale"), (dict(ws=ws.view(4)), "w_scale"),
                     (dict(out_dtype=torch.float16), "out_dtype"), (dict(gated=True), "w"),
                     (dict(y=torch.zeros(4, 130)), "y"), (dict(y_scale=xs), "y_scale"),
                     (dict(y=torch.zeros(4, 131, dtype=bf16)[:, :130]), "contiguous"), (dict(), "GPU")):
        a = dict(w=w, ws=ws, x=x, xs=xs)
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.linear_e4m3(a.pop("w"), a.pop("ws"), a.pop("x"), a.pop("xs"), **a)
    r = q4.DeviceRouting(2, 8, 2, "cpu")
    we, wse = torch.zeros(8, 64, 192).to(f8), torch.zeros(8, 1, 2)
    for kw, what in ((dict(w=we[:7]), "w"), (dict(x=x[:3]), "rows"), (dict(x=x[:0]), "rows"),
                     (dict(x=torch.zeros(6, 192).to(f8)), "T=2"), (dict(ws=wse[:7]), "w_scale"),
                     (dict(gated=True), "w"), (dict(), "GPU")):
        a = dict(w=we, ws=wse, x=x, xs=torch.zeros(6, 2))
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.experts_e4m3(a.pop("w"), a.pop("ws"), a.pop("x"), a.pop("xs"), r, **a)


def test_expert_order_binding_refuses():
    r = q4.DeviceRouting(3, 8, 2, "cpu")
    x, rows = torch.zeros(3, 128, dtype=bf16), torch.zeros(6, 128, dtype=bf16)
    for call, what in ((lambda: q4.dispatch(x[0], r), "x"), (lambda: q4.dispatch(x.float(), r), "x"),
                       (lambda: q4.dispatch(torch.zeros(4, 128, dtype=bf16), r), "T=3"),
                       (lambda: q4.dispatch(x, r, rows=rows[:5]), "rows"),
                       (lambda: q4.dispatch(x, r, e4m3=True, rows=rows), "rows"),
                       (lambda: q4.dispatch(x, r, rows_scale=torch.zeros(5, 1)), "rows_scale"),
                       (lambda: q4.dispatch(x, r), "GPU"),
                       (lambda: q4.combine(rows[:5], r), "rows"), (lambda: q4.combine(rows[0], r), "rows"),
                       (lambda: q4.combine(rows.float(), r), "rows"),
                       (lambda: q4.combine(rows, r, base=x[:2]), "base"),
                       (lambda: q4.combine(rows, r, y=x[:2]), "y"), (lambda: q4.combine(rows, r), "GPU"),
                       (lambda: q4.combine_grad(x[:2], rows, r), "tokens"),
                       (lambda: q4.combine_grad(x[:, :64], rows, r), "dy"),
                       (lambda: q4.combine_grad(x, rows, r, d_rows=rows[:4]), "d_rows"),
                       (lambda: q4.combine_grad(x, rows, r, d_w=torch.zeros(5)), "d_w"),
                       (lambda: q4.combine_grad(x, rows, r), "GPU")):
        with pytest.raises(ValueError, match=what):
            call()


def test_penalize_binding_refuses():
    l, t = torch.zeros(2, 100), torch.zeros(2, 5, dtype=i32)
    n, b = torch.zeros(2, dtype=i32), torch.zeros(2, 3)
    for kw, what in ((dict(logits=l[0]), "logits"), (dict(logits=l.half()), "logits"),
                     (dict(tokens=t[0]), "tokens"), (dict(tokens=t[:1]), "tokens"),
                     (dict(tokens=t.long()), "tokens"), (dict(n_tokens=n), "needs tokens"),
                     (dict(tokens=t, n_tokens=n[:1]), "n_tokens"),
                     (dict(tokens=t, n_prompt=n.long()), "n_prompt"),
                     (dict(repetition=torch.ones(1)), "repetition"), (dict(bias=b), "together"),
                     (dict(bias=b, bias_ids=t), "bias"), (dict(bias=b, bias_ids=t[:, :3]), "contiguous"),
                     (dict(mask=torch.zeros(2, 3, dtype=i32)), "mask"),
                     (dict(mask=torch.zeros(2, 4)), "mask"), (dict(out=l[:1]), "out"), (dict(), "GPU")):
        a = dict(logits=l)
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            q4.penalize(a.pop("logits"), **a)


def test_norm_groups_refuse():
    call = lambda flags: _abi.lib().moe_add_norm(FAKE, 2, 128, None, None, FAKE, 1e-6, flags, None,  # noqa: E731
                                                 None, None, None)
    assert call(_abi.MOE_NORM_GROUP_128) == EINVAL and b"neither" in _abi.lib().moe_last_error()
    x = torch.zeros(2, 192, dtype=bf16)
    with pytest.raises(ValueError, match="group"):
        q4.add_norm(x, x[0], e4m3=True, group=32)
    with pytest.raises(ValueError, match="y8_scale"):
        q4.add_norm(x, x[0], y8_scale=torch.zeros(3), group=128)


@pytest.mark.parametrize("shape", [(1, 64), (130, 192), (3, 128, 256), (2, 2, 65, 320)])
def test_quantize_blocks(shape):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(*shape, generator=g)
    w[..., 0, :] = 0
    codes, scale = q4.quantize_blocks(w)
    N, K = shape[-2:]
    assert codes.dtype == f8 and codes.shape == w.shape
    assert scale.shape == (*shape[:-2], -(-N // 128), -(-K // 128))
    flat = lambda t: t.reshape(-1, *t.shape[-2:])                                    # noqa: E731
    for c, s, v in zip(flat(codes), flat(scale), flat(w)):
        full = np.repeat(np.repeat(s.double().numpy(), 128, 0)[:N], 128, 1)[:, :K]
        err = np.abs(values(c) * full - v.double().numpy())
        assert (err <= np.maximum(np.abs(v.numpy()) * 2.0 ** -4, full * 2.0 ** -10) * (1 + 2 ** -20)).all()
    assert q4.quantize_blocks(torch.zeros(2, 64))[1].item() == 0
    with pytest.raises(ValueError, match="floating"):
        q4.quantize_blocks(torch.zeros(2, 64, dtype=i32))


def test_host_made_routings_are_what_the_kernels_take():
    rng = np.random.default_rng(2)
    idx, w = selections(rng, 40, 6, 3)
    r, o = device_routing(idx, w, 6, "cpu", room=2)
    assert int(r.offsets[6]) == 120 and int(r.n_tiles) == sum(-(-int(c) // 128) for c in o["counts"])
    assert np.array_equal(np.sort(r.inv_perm[:120].numpy()), np.arange(120))
    x, s = quantised_rows(rng, 5, 192)
    assert x.shape == (5, 192) and s.shape == (5, 2)


def test_own_buffers_are_allocated_with_the_calls_stream_current(monkeypatch):
    """(on the CPU: every allocation happens inside the stream's context; the calls are
    refused afterwards, because the tensors are not on the GPU)"""
    import contextlib
    import types

    from torch.utils._python_dispatch import TorchDispatchMode

    class Allocations(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.seen, self.active = [], False

        def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
            if "empty" in func.overloadpacket.__name__ or "zeros" in func.overloadpacket.__name__:
                self.seen.append(self.active)
            return func(*args, **(kwargs or {}))

    r = q4.DeviceRouting(2, 8, 2, "cpu")
    x, rows = torch.zeros(2, 128, dtype=bf16), torch.zeros(4, 128, dtype=bf16)
    x8, xs = torch.zeros(4, 128).to(f8), torch.zeros(4, 1)
    w, ws = torch.zeros(8, 2, 64, 128).to(f8), torch.zeros(8, 2, 1, 1)
    calls = [(lambda s: q4.linear_e4m3(w[0], ws[0], x8, xs, gated=True, stream=s), 2),
             (lambda s: q4.linear_e4m3(w[0, 0], ws[0, 0], x8, xs, stream=s), 1),
             (lambda s: q4.experts_e4m3(w, ws, x8, xs, r, gated=True, stream=s), 2),
             (lambda s: q4.dispatch(x, r, e4m3=True, stream=s), 2),
             (lambda s: q4.combine(rows, r, stream=s), 1),
             (lambda s: q4.combine_grad(x, rows, r, stream=s), 2),
             (lambda s: q4.penalize(torch.zeros(2, 9), stream=s), 1)]
    mode, stream = Allocations(), types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0)

    @contextlib.contextmanager
    def current(s):
        mode.active = s is stream
        yield
        mode.active = False

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    for call, n in calls:
        mode.seen.clear()
        if n == 1 and call is calls[-1][0]:
            l = torch.zeros(2, 9)
            call = lambda s: q4.penalize(l, stream=s)                                # noqa: E731
        with mode, pytest.raises(ValueError, match="GPU"):
            call(stream)
        assert len(mode.seen) >= n and all(mode.seen)
