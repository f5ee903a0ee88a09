"""Python binding of libq4moe.so, the gfx950 routed-MoE Q4 FFN layer.

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI of include/q4moe.h.  PyTorch supplies device memory and the
stream.  There is no fallback: if the library is missing, loading raises.

Calls launch on the current stream or on `stream`.  What a call allocates itself
(outputs, routings, workspaces) is allocated on the stream it launches on; tensors
that are given to it have to be ready on that stream, and the weights of a layer or
head to be kept until the work is done, as everywhere in torch.

    layer = DeviceLayer.from_host(L)           # L: dict of numpy arrays
    r = route(layer, x)                        # x: bf16 [T, d] on the GPU
    y = prefill(layer, x, r)                   # bf16 [T, d]
    y1 = decode(layer, x1, ws)                 # one token
    lm = DeviceLmHead.from_host(head, embed)     # V x d output head, embedding
    logits, tok, _ = lm_argmax(lm, h, lm_workspace(lm), x_next=x_in)  # greedy token

The operators around the layer:

    y, _, _ = add_norm(x, w, residual, residual_out=residual)  # bf16 [T, d]
    r = route_scored(layer, y, RouterSpec(score="sigmoid", balance=b))
    y = decode_tokens(layer, y, ws, routing=r, routing_in=True)  # or prefill(layer, y, r)
    logits = linear(q, scale, bias, h)                         # fp32 [T, N], T <= 64
    logits = penalize(logits, tokens=history, repetition=1.1, mask=grammar, out=logits)
    token, prob, _ = sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)

Experts in 8 bits (e4m3, a scale per token and 128 columns and per 128 x 128 weights):

    w13, s13 = quantize_blocks(gate_up)        # [E, 2, I, d], once
    rows, rows_s = dispatch(x, r, e4m3=True)   # expert-sorted rows
    h, h_s = experts_e4m3(w13, s13, rows, rows_s, r, gated=True)
    y = combine(experts_e4m3(w2, s2, h, h_s, r), r, base=shared)
    logits = linear_e4m3(w, s, *add_norm(x, w, e4m3=True, group=128)[1:])

No call records an autograd graph.  dispatch and combine have gradients, as calls of their own
(combine unweighted, combine_grad); where a graph is being recorded they refuse tensors that
require a gradient (call them under torch.no_grad(), or from a torch.autograd.Function).
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch

from . import _abi

MOE_LOGITS_IN = _abi.MOE_LOGITS_IN
MAX_DECODE_TOKENS = _abi.MOE_MAX_DECODE_TOKENS
MAX_LINEAR_TOKENS = _abi.MOE_MAX_LINEAR_TOKENS
BLOCK_ROWS = _abi.MOE_BLOCK_ROWS
TILE_ROWS = _abi.MOE_TILE_ROWS
MATS = ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        lib = _abi.lib()
        self.code = code
        msg = lib.moe_strerror(code).decode()
        detail = lib.moe_last_error().decode()
        super().__init__(f"{where}: {msg} ({code}): {detail}")


def _check(code: int, where: str):
    if code != 0:
        raise MoEError(code, where)


def _stream() -> int:
    return int(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name: str, dtype, n: int):
    """The C ABI sees only pointers, so the binding checks what the kernels will
    touch: a contiguous tensor of `dtype` with at least n elements (and, through
    _on_gpu, in device memory)."""
    if t is not None and t.dtype is dtype and t.numel() >= n and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: {t.numel()} elements, the call touches {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU")


def _on_stream(call, args: dict):
    """call(**args) with args["stream"] current.  A call's own buffers (outputs,
    routings, workspaces) then come from the stream it launches on: memory from another
    stream's pool may still be in use by that stream's queued work, its fills are not
    ordered before the call's kernels, and once dropped it goes to that stream's next
    tensor, which does not wait for them either."""
    stream = args.pop("stream")
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(**args)
    _used_on(stream, *args.values())
    _used_on(caller, *(out if isinstance(out, tuple) else (out,)))  # after a wait
    return out


def _used_on(stream, *values):
    """Keeps the memory of the tensors among the values from being handed out again
    before the work that is now on `stream` is done."""
    for v in values:
        if isinstance(v, DeviceRouting):
            _used_on(stream, *(getattr(v, f) for f, _ in _abi.Routing._fields_))
        elif isinstance(v, RouterSpec):
            _used_on(stream, v.balance)
        elif isinstance(v, torch.Tensor) and v.is_cuda:
            v.record_stream(stream)


def _dev(a: np.ndarray, device) -> torch.Tensor:
    a = np.ascontiguousarray(a)
    view = {np.dtype(np.uint32): np.int32, np.dtype(np.uint16): np.int16}.get(a.dtype, a.dtype)
    return torch.from_numpy(a.view(view)).to(device)


class DeviceLayer:
    """One layer's weights in device memory plus the moe_layer struct pointing at them."""

    def __init__(self, d, inter, n_experts, top_k, tensors: dict):
        self.d, self.inter, self.n_experts, self.top_k = d, inter, n_experts, top_k
        self.t = tensors
        mats = {m: _abi.Q4Mat(_ptr(tensors[m + "_q"]), _ptr(tensors[m + "_s"]),
                              _ptr(tensors[m + "_b"])) for m in MATS}
        self.struct = _abi.Layer(d, inter, n_experts, top_k, _ptr(tensors["w_router"]),
                                 _ptr(tensors.get("router_bias")), *[mats[m] for m in MATS])

    @classmethod
    def from_host(cls, L: dict, device="cuda"):
        t = {}
        for m in MATS:
            for suf in ("_q", "_s", "_b"):
                t[m + suf] = _dev(L[m + suf], device)
        t["w_router"] = _dev(L["w_router"].astype(np.float32), device)
        if L.get("router_bias") is not None:
            t["router_bias"] = _dev(L["router_bias"].astype(np.float32), device)
        return cls(L["d"], L["inter"], L["n_experts"], L["top_k"], t)

    def weight_bytes(self) -> int:
        return sum(v.numel() * v.element_size() for k, v in self.t.items()
                   if k.endswith(("_q", "_s", "_b")))


class DeviceRouting:
    """Device arrays of moe_routing for up to T tokens."""

    def __init__(self, T: int, n_experts: int, top_k: int, device="cuda"):
        lib = _abi.lib()
        i32 = dict(dtype=torch.int32, device=device)
        self.T, self.E, self.k = T, n_experts, top_k
        self.logits = torch.zeros((T, n_experts), dtype=torch.float32, device=device)
        self.topk_idx = torch.zeros((T, top_k), **i32)
        self.topk_w = torch.zeros((T, top_k), dtype=torch.float32, device=device)
        self.counts = torch.zeros(n_experts, **i32)
        self.offsets = torch.zeros(n_experts + 1, **i32)
        self.perm = torch.zeros(T * top_k, **i32)
        self.inv_perm = torch.zeros(T * top_k, **i32)
        nb = lib.moe_block_map_capacity(T, top_k, n_experts, BLOCK_ROWS)
        nt = lib.moe_block_map_capacity(T, top_k, n_experts, TILE_ROWS)
        self.block_map = torch.zeros((nb, 2), **i32)
        self.n_blocks = torch.zeros(1, **i32)
        self.tile_map = torch.zeros((nt, 2), **i32)
        self.n_tiles = torch.zeros(1, **i32)
        n_blk = (T + _abi.MOE_ROUTE_BLOCK - 1) // _abi.MOE_ROUTE_BLOCK
        self.blk_counts = torch.zeros((n_blk, n_experts), **i32)
        self.struct = _abi.Routing(*[_ptr(getattr(self, f)) for f, _ in _abi.Routing._fields_])


def workspace_bytes(layer: DeviceLayer, T: int) -> int:
    n = _abi.lib().moe_workspace_bytes(C.addressof(layer.struct), T)
    if n == 0:
        raise MoEError(_abi.MOE_EINVAL, "moe_workspace_bytes")
    return int(n)


def workspace(layer: DeviceLayer, T: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for moe_prefill (T tokens) and moe_decode."""
    return torch.zeros(workspace_bytes(layer, T), dtype=torch.uint8, device=device)


def route(layer: DeviceLayer, x: torch.Tensor, routing: DeviceRouting | None = None,
          logits_in: bool = False, stream=None) -> DeviceRouting:
    if stream is not None:
        return _on_stream(route, locals())
    T = x.shape[0]
    r = routing or DeviceRouting(T, layer.n_experts, layer.top_k, x.device)
    flags = MOE_LOGITS_IN if logits_in else 0
    if not logits_in:
        _need(x, "x", torch.bfloat16, T * layer.d)
    _need(r.logits, "routing.logits", torch.float32, T * layer.n_experts)
    _need(r.perm, "routing.perm", torch.int32, T * layer.top_k)
    _on_gpu(x=None if logits_in else x, logits=r.logits)
    _check(_abi.lib().moe_route(C.addressof(layer.struct), _ptr(x), T, flags, C.addressof(r.struct),
                                _stream()), "moe_route")
    return r


class RouterSpec:
    """How route_scored scores and selects: score "softmax" or "sigmoid"; balance (fp32
    [E] on the GPU, or None) is added to the scores for the selection only; the
    experts fall into n_groups runs, of which the top_groups best by the sum of
    their group_top (1 or 2) largest values take part; renorm divides the weights by
    their sum; scale multiplies them."""

    def __init__(self, score: str = "softmax", n_groups: int = 1, top_groups: int = 1,
                 group_top: int = 1, renorm: bool = True, scale: float = 1.0,
                 balance: torch.Tensor | None = None):
        kinds = {"softmax": _abi.MOE_SCORE_SOFTMAX, "sigmoid": _abi.MOE_SCORE_SIGMOID}
        if score not in kinds:
            raise ValueError(f"score must be one of {sorted(kinds)}, not {score!r}")
        if balance is not None:
            _need(balance, "balance", torch.float32, 1)
        self.balance = balance  # keep the tensor alive
        self.struct = _abi.RouterSpec(kinds[score], n_groups, top_groups, group_top, int(renorm),
                                      scale, _ptr(balance))


def route_scored(layer: DeviceLayer, x: torch.Tensor | None, spec: RouterSpec,
                 routing: DeviceRouting | None = None, logits_in: bool = False,
                 stream=None) -> DeviceRouting:
    """Routing with the scores and the selection of `spec`.  Follow it with prefill,
    or with decode / decode_tokens and routing_in=True.  With logits_in the T =
    routing.T rows of routing.logits are routed; x is not used."""
    if stream is not None:
        return _on_stream(route_scored, locals())
    if logits_in:
        if routing is None:
            raise ValueError("logits_in needs a routing that holds the logits")
        T = routing.T
    else:
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, T * layer.d)
        if routing is None:
            routing = DeviceRouting(T, layer.n_experts, layer.top_k, x.device)
    r = routing
    if r.T < T or r.E != layer.n_experts or r.k != layer.top_k:
        raise ValueError(f"routing is for T={r.T} E={r.E} k={r.k}, the call for T={T} "
                         f"E={layer.n_experts} k={layer.top_k}")
    if spec.balance is not None:
        _need(spec.balance, "balance", torch.float32, layer.n_experts)
    s = _launch_on("route_scored", x=None if logits_in else x, logits=r.logits,
                   balance=spec.balance)
    _check(_abi.lib().moe_route_scored(C.addressof(layer.struct), None if logits_in else _ptr(x), T,
                                       MOE_LOGITS_IN if logits_in else 0, C.addressof(spec.struct),
                                       C.addressof(r.struct), s), "moe_route_scored")
    return r


_ITEM_ROWS_FLAGS = {128: 0, 64: _abi.MOE_ITEM_ROWS_64, 32: _abi.MOE_ITEM_ROWS_32,
                    16: _abi.MOE_ITEM_ROWS_16}


def prefill(layer: DeviceLayer, x: torch.Tensor, routing: DeviceRouting,
            ws: torch.Tensor | None = None, y: torch.Tensor | None = None,
            stream=None, item_rows: int = 128) -> torch.Tensor:
    """moe_prefill (item_rows = 128) or moe_prefill_ex with the gate/up work-item
    height item_rows (64, 32 or 16)."""
    if stream is not None:
        return _on_stream(prefill, locals())
    if item_rows not in _ITEM_ROWS_FLAGS:
        raise ValueError(f"item_rows must be one of 128, 64, 32, 16, not {item_rows}")
    T = x.shape[0]
    if ws is None:
        ws = workspace(layer, T, x.device)
    if y is None:
        y = torch.empty((T, layer.d), dtype=torch.bfloat16, device=x.device)
    _need(x, "x", torch.bfloat16, T * layer.d)
    _need(y, "y", torch.bfloat16, T * layer.d)
    _need(routing.perm, "routing.perm", torch.int32, T * layer.top_k)
    _on_gpu(x=x, y=y, ws=ws, perm=routing.perm)
    if item_rows == 128:
        _check(_abi.lib().moe_prefill(C.addressof(layer.struct), _ptr(x), T,
                                      C.addressof(routing.struct), _ptr(ws), ws.numel(), _ptr(y),
                                      _stream()),
               "moe_prefill")
    else:
        _check(_abi.lib().moe_prefill_ex(C.addressof(layer.struct), _ptr(x), T,
                                         C.addressof(routing.struct), _ptr(ws), ws.numel(),
                                         _ptr(y), _ITEM_ROWS_FLAGS[item_rows], _stream()),
               "moe_prefill_ex")
    return y


def _decode_flags(layer, T: int, routing, logits_in: bool, routing_in: bool) -> int:
    if routing is not None:
        _need(routing.logits, "routing.logits", torch.float32, T * layer.n_experts)
        _need(routing.topk_idx, "routing.topk_idx", torch.int32, T * layer.top_k)
        _need(routing.topk_w, "routing.topk_w", torch.float32, T * layer.top_k)
    if routing_in:
        if routing is None:
            raise ValueError("routing_in needs a routing")
        # rows of another length would be read across each other
        if routing.E != layer.n_experts or routing.k != layer.top_k:
            raise ValueError(f"the routing is for E={routing.E} k={routing.k}, the layer has "
                             f"E={layer.n_experts} k={layer.top_k}")
        _on_gpu(**{"routing.topk_idx": routing.topk_idx, "routing.topk_w": routing.topk_w})
    return (MOE_LOGITS_IN if logits_in else 0) | (_abi.MOE_ROUTING_IN if routing_in else 0)


def decode(layer: DeviceLayer, x: torch.Tensor, ws: torch.Tensor, y: torch.Tensor | None = None,
           routing: DeviceRouting | None = None, logits_in: bool = False,
           stream=None, routing_in: bool = False) -> torch.Tensor:
    """The layer for one token.  routing_in: the selection in routing (from route or
    route_scored) is used instead of the layer's own routing."""
    if stream is not None:
        return _on_stream(decode, locals())
    if y is None:
        y = torch.empty((1, layer.d), dtype=torch.bfloat16, device=x.device)
    rs = C.addressof(routing.struct) if routing is not None else None
    _need(x, "x", torch.bfloat16, layer.d)
    _need(y, "y", torch.bfloat16, layer.d)
    flags = _decode_flags(layer, 1, routing, logits_in, routing_in)
    _on_gpu(x=x, y=y, ws=ws)
    _check(_abi.lib().moe_decode(C.addressof(layer.struct), _ptr(x), flags, rs, _ptr(ws), ws.numel(),
                                 _ptr(y), _stream()), "moe_decode")
    return y


def decode_tokens(layer: DeviceLayer, x: torch.Tensor, ws: torch.Tensor,
                  y: torch.Tensor | None = None, routing: DeviceRouting | None = None,
                  logits_in: bool = False, stream=None,
                  routing_in: bool = False) -> torch.Tensor:
    """The decode layer for T = x.shape[0] tokens (1 <= T <= MAX_DECODE_TOKENS).
    routing_in: as decode's."""
    if stream is not None:
        return _on_stream(decode_tokens, locals())
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, layer.d), dtype=torch.bfloat16, device=x.device)
    rs = C.addressof(routing.struct) if routing is not None else None
    _need(x, "x", torch.bfloat16, T * layer.d)
    _need(y, "y", torch.bfloat16, T * layer.d)
    flags = _decode_flags(layer, T, routing, logits_in, routing_in)
    _on_gpu(x=x, y=y, ws=ws)
    _check(_abi.lib().moe_decode_tokens(C.addressof(layer.struct), _ptr(x), T, flags, rs, _ptr(ws),
                                        ws.numel(), _ptr(y), _stream()), "moe_decode_tokens")
    return y


def dequant(q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor, stream=None) -> torch.Tensor:
    """bf16 [N, K] from one Q4 matrix (q int32 [N, K/8], scale/bias bf16 bits [N, K/64])."""
    if stream is not None:
        return _on_stream(dequant, locals())
    N, K = q.shape[0], q.shape[1] * 8
    out = torch.empty((N, K), dtype=torch.bfloat16, device=q.device)
    m = _abi.Q4Mat(_ptr(q), _ptr(scale), _ptr(bias))
    _check(_abi.lib().moe_dequant(C.addressof(m), N, K, _ptr(out), _stream()), "moe_dequant")
    return out


class DeviceLmHead:
    """An output head and embedding table (V x d Q4 each) in device memory, plus
    the moe_lm_head struct pointing at them."""

    def __init__(self, V: int, d: int, head: dict, embed: dict | None):
        self.V, self.d = V, d
        self.head, self.embed = head, embed  # keep the tensors alive

        def mat(m):
            return _abi.Q4Mat() if m is None else _abi.Q4Mat(_ptr(m["q"]), _ptr(m["scale"]),
                                                              _ptr(m["bias"]))
        self.struct = _abi.LmHead(V, d, mat(head), mat(embed))

    @classmethod
    def from_host(cls, head: dict, embed: dict | None = None, device="cuda"):
        """head / embed: dicts of numpy q uint32 [V, d/8], scale, bias uint16 [V, d/64]."""
        V, d = head["q"].shape[0], head["q"].shape[1] * 8
        dev = lambda m: None if m is None else {k: _dev(m[k], device) for k in ("q", "scale", "bias")}
        return cls(V, d, dev(head), dev(embed))


def lm_workspace(lm: DeviceLmHead, device="cuda") -> torch.Tensor:
    n = _abi.lib().moe_lm_workspace_bytes(C.addressof(lm.struct))
    if n == 0:
        raise MoEError(_abi.MOE_EINVAL, "moe_lm_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def lm_argmax(lm: DeviceLmHead, x: torch.Tensor | None, ws: torch.Tensor,
              logits: torch.Tensor | None = None, token: torch.Tensor | None = None,
              x_next: torch.Tensor | None = None, logits_in: bool = False, stream=None):
    """Greedy token hand-off: (logits fp32 [V], token int32 [1], x_next or None).
    With logits_in the given logits are read instead of computed from x."""
    if stream is not None:
        return _on_stream(lm_argmax, locals())
    dev = ws.device
    if logits is None:
        logits = torch.empty(lm.V, dtype=torch.float32, device=dev)
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=dev)
    flags = MOE_LOGITS_IN if logits_in else 0
    if not logits_in:
        _need(x, "x", torch.bfloat16, lm.d)
    _need(logits, "logits", torch.float32, lm.V)
    _need(token, "token", torch.int32, 1)
    if x_next is not None:
        _need(x_next, "x_next", torch.bfloat16, lm.d)
    _on_gpu(x=None if logits_in else x, logits=logits, token=token, x_next=x_next, ws=ws)
    _check(_abi.lib().moe_lm_argmax(C.addressof(lm.struct), _ptr(x), flags, _ptr(logits),
                                    _ptr(token), _ptr(x_next), _ptr(ws), ws.numel(),
                                    _stream()), "moe_lm_argmax")
    return logits, token, x_next


# The current stream's handle without building a stream object (2.5 us of a call), and the
# current device without asking whether the GPU is initialised (its tensors are at hand).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _not_on_one_gpu(where: str, tensors: dict):
    """The error of _launch_on for tensors that are not all on one GPU."""
    dev = -1
    for name, t in tensors.items():
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{name} must be on the GPU")
        if dev >= 0 and d != dev:
            raise ValueError(f"{where}: {name} is on cuda:{d}, other arguments on cuda:{dev}")
        dev = d


def _launch_on(where: str, **tensors) -> int:
    """The current stream's handle for a call whose tensors are `tensors` (None: absent).
    All of them have to be on one GPU, and that GPU has to be the current one, because
    the library launches on the current device."""
    dev = -1
    for t in tensors.values():
        if t is not None:
            d = t.get_device()
            if d != dev or d < 0:
                if d < 0 or dev >= 0:
                    _not_on_one_gpu(where, tensors)
                dev = d
    if dev != _current_device():
        raise ValueError(f"{where}: the tensors are on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return _raw_stream(dev)


def sample_workspace(B: int, V: int, device="cuda") -> torch.Tensor:
    """A workspace for sample: B rows of V logits."""
    n = _abi.lib().moe_sample_workspace_bytes(V, B)
    if n == 0:
        raise MoEError(_abi.MOE_EINVAL, "moe_sample_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           lm: DeviceLmHead | None = None, token: torch.Tensor | None = None,
           prob: torch.Tensor | None = None, x_next: torch.Tensor | None = None,
           ws: torch.Tensor | None = None, stream=None):
    """One token for each row of logits [B, V] (fp32) from uniform numbers u [B] (fp32):
    (token int32 [B], prob fp32 [B], x_next or None).  temperature (0: greedy), top_k
    (0: off), top_p (1: off) and min_p (0: off) are numbers for all rows or tensors [B]
    on the GPU (fp32; top_k int32).  x_next [B, d] needs lm, whose embedding rows it
    gets.  ws: sample_workspace(B, V) or larger."""
    if stream is not None:
        return _on_stream(sample, locals())
    if logits.dim() != 2:
        raise ValueError(f"logits must be [B, V], not {tuple(logits.shape)}")
    B, V = logits.shape
    _need(logits, "logits", torch.float32, B * V)
    _need(u, "u", torch.float32, B)
    p = _abi.Sampling(_ptr(u))
    rows = {"u": u}
    for name, v, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(v, torch.Tensor):
            _need(v, name, dt, B)
            rows[name] = v
            setattr(p, name, v.data_ptr())
        else:
            if dt == torch.int32 and not -2**31 <= v < 2**31:
                raise ValueError(f"{name}: {v} is not an int32")
            setattr(p, name + "_all", v)
    if token is None:
        token = logits.new_empty(B, dtype=torch.int32)
    if prob is None:
        prob = logits.new_empty(B)
    _need(token, "token", torch.int32, B)
    _need(prob, "prob", torch.float32, B)
    if x_next is not None:
        if lm is None or lm.V != V or lm.embed is None:
            raise ValueError(f"x_next needs an lm head of V={V} with an embedding table")
        _need(x_next, "x_next", torch.bfloat16, B * lm.d)
        head = lm.struct
    else:
        head = _abi.LmHead(V)
    if ws is None:
        ws = sample_workspace(B, V, logits.device)
    _need(ws, "ws", torch.uint8, 1)
    s = _launch_on("sample", logits=logits, token=token, prob=prob, x_next=x_next, ws=ws,
                   **rows)
    _check(_abi.lib().moe_sample(C.addressof(head), _ptr(logits), B, C.addressof(p), _ptr(token),
                                 _ptr(prob), _ptr(x_next), _ptr(ws), ws.numel(), s), "moe_sample")
    return token, prob, x_next


def linear(q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor, x: torch.Tensor,
           out_dtype: torch.dtype = torch.float32, y: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """y [T, N] = x [T, K] times the transposed Q4 matrix (q int32 [N, K/8], scale and
    bias bf16 or their bits [N, K/64]), 1 <= T <= MAX_LINEAR_TOKENS; out_dtype fp32
    or bf16."""
    if stream is not None:
        return _on_stream(linear, locals())
    if x.dim() != 2 or q.dim() != 2:
        raise ValueError(f"x must be [T, K] and q [N, K/8], not {tuple(x.shape)}, {tuple(q.shape)}")
    T, K = x.shape
    N = q.shape[0]
    if q.shape[1] * 8 != K:
        raise ValueError(f"q has {q.shape[1] * 8} columns, x has {K}")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, not {out_dtype}")
    if y is None:
        y = x.new_empty((T, N), dtype=out_dtype)
    _need(x, "x", torch.bfloat16, T * K)
    _need(q, "q", torch.int32, N * K // 8)
    for name, t in (("scale", scale), ("bias", bias)):
        _need(t, name, torch.int16 if t.dtype == torch.int16 else torch.bfloat16, N * (K // 64))
    _need(y, "y", out_dtype, T * N)
    s = _launch_on("linear", q=q, scale=scale, bias=bias, x=x, y=y)
    m = _abi.Q4Mat(_ptr(q), _ptr(scale), _ptr(bias))
    _check(_abi.lib().moe_linear(C.addressof(m), N, K, _ptr(x), T,
                                 _abi.MOE_OUT_BF16 if out_dtype == torch.bfloat16 else 0, _ptr(y),
                                 s), "moe_linear")
    return y


def _blocks(n: int, size: int = _abi.MOE_E4M3_BLOCK) -> int:
    return -(-n // size)


def add_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
             eps: float = 1e-6, plus_one: bool = False, residual_out: torch.Tensor | None = None,
             y: torch.Tensor | None = None, e4m3: bool = False, y8: torch.Tensor | None = None,
             y8_scale: torch.Tensor | None = None, stream=None, group: int = 64):
    """Residual addition and RMS norm of the rows of x [T, d] (bf16): (y, y8, y8_scale).

    residual: bf16 or fp32 [T, d]; x + residual goes to residual_out (which may be
    residual itself; None: not stored).  plus_one: the weight used is weight + 1.
    y (bf16) is written when given, and by default when no 8-bit output is asked
    for; e4m3=True (or y8 and y8_scale given) asks for e4m3 codes [T, d] with one
    fp32 scale per `group` columns [T, ceil(d / group)], 64 or 128 (what linear_e4m3
    takes)."""
    if stream is not None:
        return _on_stream(add_norm, locals())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], not {tuple(x.shape)}")
    T, d = x.shape
    flags = _abi.MOE_NORM_PLUS_ONE if plus_one else 0
    if group not in (64, 128):
        raise ValueError(f"group must be 64 or 128, not {group}")
    if group == 128:
        flags |= _abi.MOE_NORM_GROUP_128
    _need(x, "x", torch.bfloat16, T * d)
    _need(weight, "weight", torch.bfloat16, d)
    if residual is not None:
        rt = torch.float32 if residual.dtype == torch.float32 else torch.bfloat16
        _need(residual, "residual", rt, T * d)
        if residual_out is not None:
            _need(residual_out, "residual_out", rt, T * d)
        if rt == torch.float32:
            flags |= _abi.MOE_NORM_RESIDUAL_FLOAT
    e4m3 = e4m3 or y8 is not None or y8_scale is not None
    if e4m3:
        if y8 is None:
            y8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        if y8_scale is None:
            y8_scale = x.new_empty((T, _blocks(d, group)), dtype=torch.float32)
        _need(y8, "y8", torch.float8_e4m3fn, T * d)
        _need(y8_scale, "y8_scale", torch.float32, T * _blocks(d, group))
    elif y is None:
        y = torch.empty_like(x)
    if y is not None:
        _need(y, "y", torch.bfloat16, T * d)
    s = _launch_on("add_norm", x=x, weight=weight, residual=residual,
                   residual_out=residual_out, y=y, y8=y8, y8_scale=y8_scale)
    _check(_abi.lib().moe_add_norm(_ptr(x), T, d, _ptr(residual), _ptr(residual_out), _ptr(weight),
                                   eps, flags, _ptr(y), _ptr(y8), _ptr(y8_scale), s),
           "moe_add_norm")
    return y, y8, y8_scale


def quantize_blocks(w: torch.Tensor):
    """e4m3 codes of matrices w [..., N, K] (any floating type) and fp32 scales
    [..., ceil(N / 128), ceil(K / 128)], max |w| / 448 of each 128 x 128 block: what
    linear_e4m3 and experts_e4m3 take.  Done once, when weights are loaded (elementary
    torch operations)."""
    B = _abi.MOE_E4M3_BLOCK
    if w.dim() < 2 or not w.is_floating_point():
        raise ValueError(f"w must be floating [..., N, K], not {w.dtype} {tuple(w.shape)}")
    N, K = w.shape[-2:]
    nb, kb = _blocks(N), _blocks(K)
    g = torch.nn.functional.pad(w.float(), (0, kb * B - K, 0, nb * B - N))
    g = g.reshape(*w.shape[:-2], nb, B, kb, B)
    scale = g.abs().amax((-3, -1)) / 448.0
    s = scale[..., :, None, :, None]
    codes = torch.where(s > 0, g / s, 0.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    codes = codes.reshape(*w.shape[:-2], nb * B, kb * B)[..., :N, :K]
    return codes.contiguous(), scale.contiguous()


def _product(where, w, w_scale, x, x_scale, lead, rows, out_dtype, gated, y, y_scale):
    """Checks and outputs shared by the 8-bit products: the C call's matrix, N (both parts
    of a gated matrix), K, flags, y, y_scale."""
    if gated:
        lead, out_dtype = lead + (2,), torch.float8_e4m3fn
    elif out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, not {out_dtype}")
    shape, given = w.shape, x.shape
    if len(given) != 2 or len(shape) != len(lead) + 2 or shape[:-2] != lead:
        raise ValueError(f"{where}: x must be [rows, K] and w {[*lead, 'N', 'K']}, not "
                         f"{tuple(given)}, {tuple(shape)}")
    N, K = shape[-2:]
    if given[1] != K:
        raise ValueError(f"{where}: w has {K} columns, x has {given[1]}")
    kb, nb = (K + 127) >> 7, (N + 127) >> 7
    # (a scale per 64 columns has enough elements too, and would be read as another's)
    if x_scale.shape[-1:] != (kb,) or w_scale.shape[-2:] != (nb, kb):
        raise ValueError(f"{where}: x_scale must be [rows, {kb}] and w_scale {[*lead, nb, kb]}, not "
                         f"{tuple(x_scale.shape)}, {tuple(w_scale.shape)}")
    mats = 1
    for n in lead:
        mats *= n
    _need(x, "x", torch.float8_e4m3fn, rows * K)
    _need(x_scale, "x_scale", torch.float32, rows * kb)
    _need(w, "w", torch.float8_e4m3fn, mats * N * K)
    _need(w_scale, "w_scale", torch.float32, mats * nb * kb)
    if y is None:
        y = x.new_empty((rows, N), dtype=out_dtype)
    else:
        _need(y, "y", out_dtype, rows * N)
    if gated:
        if y_scale is None:
            y_scale = x_scale.new_empty((rows, nb))
        else:
            _need(y_scale, "y_scale", torch.float32, rows * nb)
    elif y_scale is not None:
        raise ValueError("y_scale is of gated products")
    flags = (_abi.MOE_GATED if gated else
             _abi.MOE_OUT_BF16 if out_dtype == torch.bfloat16 else 0)
    return _abi.E4m3Mat(w.data_ptr(), w_scale.data_ptr()), N * (2 if gated else 1), K, flags, y, y_scale


def linear_e4m3(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                out_dtype: torch.dtype = torch.bfloat16, gated: bool = False,
                y: torch.Tensor | None = None, y_scale: torch.Tensor | None = None, stream=None):
    """y [T, N] = x times the transposed matrix w, both e4m3: x [T, K] with x_scale
    [T, ceil(K / 128)], w [N, K] with w_scale [ceil(N / 128), ceil(K / 128)]; out_dtype
    bf16 or fp32.  gated: w is [2, I, K] (gate, up) with w_scale [2, ceil(I / 128), ...],
    and (y e4m3 [T, I], y_scale [T, ceil(I / 128)]) of silu(gate) * up is returned.  In bf16
    from T = 128 on, small products next to large ones that cancel may be lost: fp32 keeps them."""
    if stream is not None:
        return _on_stream(linear_e4m3, locals())
    T = x.shape[0]
    m, N, K, flags, y, y_scale = _product("linear_e4m3", w, w_scale, x, x_scale, (), T, out_dtype,
                                          gated, y, y_scale)
    s = _launch_on("linear_e4m3", w=w, w_scale=w_scale, x=x, x_scale=x_scale, y=y, y_scale=y_scale)
    _check(_abi.lib().moe_linear_scaled(C.addressof(m), N, K, x.data_ptr(), x_scale.data_ptr(), T,
                                        flags, y.data_ptr(), _ptr(y_scale), s), "moe_linear_scaled")
    return (y, y_scale) if gated else y


def _routed(where: str, routing: DeviceRouting, rows: int | None = None, T: int | None = None) -> int:
    """T of a call on expert rows (T * k of them) or tokens, which the routing has to hold."""
    if rows is not None:
        if rows % routing.k or rows == 0:
            raise ValueError(f"{where}: {rows} rows, the routing has {routing.k} for each token")
        if T is not None and T * routing.k != rows:
            raise ValueError(f"{where}: {rows} rows for {T} tokens of {routing.k} each")
        T = rows // routing.k
    if T > routing.T:
        raise ValueError(f"{where}: the routing is for T={routing.T}, the call for T={T}")
    return T


def experts_e4m3(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                 routing: DeviceRouting, out_dtype: torch.dtype = torch.bfloat16,
                 gated: bool = False, y: torch.Tensor | None = None,
                 y_scale: torch.Tensor | None = None, stream=None):
    """linear_e4m3 over the expert-sorted rows of a routing (dispatch's), with a matrix per
    expert: x [T * k, K], w [E, N, K] (gated: [E, 2, I, K]), the scales likewise.  What it says
    of T = 128 is so for 128 rows of an expert on average, T * k >= 128 * E."""
    if stream is not None:
        return _on_stream(experts_e4m3, locals())
    rows = x.shape[0]
    T = _routed("experts_e4m3", routing, rows)
    m, N, K, flags, y, y_scale = _product("experts_e4m3", w, w_scale, x, x_scale, (routing.E,),
                                          rows, out_dtype, gated, y, y_scale)
    s = _launch_on("experts_e4m3", w=w, w_scale=w_scale, x=x, x_scale=x_scale, y=y, y_scale=y_scale,
                   offsets=routing.offsets)
    _check(_abi.lib().moe_experts_scaled(C.addressof(m), routing.E, N, K, _ptr(x), _ptr(x_scale), T,
                                         routing.k, C.addressof(routing.struct), flags, _ptr(y),
                                         _ptr(y_scale), s), "moe_experts_scaled")
    return (y, y_scale) if gated else y


def _no_graph(where: str, gradient: str, **tensors):
    """Refuses inputs whose gradient would be lost unseen."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{where}: {name} requires a gradient, and the call records no graph: call "
                             f"it under torch.no_grad() or from a torch.autograd.Function ({gradient})")


def dispatch(x: torch.Tensor, routing: DeviceRouting, e4m3: bool = False,
             rows: torch.Tensor | None = None, rows_scale: torch.Tensor | None = None, stream=None):
    """Token rows x [T, d] (bf16) in expert order, k of each: (rows [T * k, d], None), or
    with e4m3 (or rows_scale given) codes and a scale per 128 columns [T * k, ceil(d / 128)].
    Its gradient is combine(d_rows, routing, weighted=False)."""
    if stream is not None:
        return _on_stream(dispatch, locals())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], not {tuple(x.shape)}")
    T, d = x.shape
    _routed("dispatch", routing, T=T)
    n = T * routing.k
    e4m3 = e4m3 or rows_scale is not None
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    if rows is None:
        rows = x.new_empty((n, d), dtype=dt)
    if e4m3 and rows_scale is None:
        rows_scale = x.new_empty((n, _blocks(d)), dtype=torch.float32)
    _need(x, "x", torch.bfloat16, T * d)
    _need(rows, "rows", dt, n * d)
    if e4m3:
        _need(rows_scale, "rows_scale", torch.float32, n * _blocks(d))
    _no_graph("dispatch", "its gradient is combine(d_rows, routing, weighted=False)", x=x)
    s = _launch_on("dispatch", x=x, rows=rows, rows_scale=rows_scale, inv_perm=routing.inv_perm)
    _check(_abi.lib().moe_dispatch(_ptr(x), T, routing.k, d, C.addressof(routing.struct),
                                   _ptr(rows), _ptr(rows_scale), s), "moe_dispatch")
    return rows, rows_scale


def combine(rows: torch.Tensor, routing: DeviceRouting, weighted: bool = True,
            base: torch.Tensor | None = None, y: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """y [T, d] (bf16): the sum over every token's slots of its expert rows [T * k, d] (bf16)
    times routing.topk_w (weighted=False: unweighted), plus base [T, d] (bf16)."""
    if stream is not None:
        return _on_stream(combine, locals())
    if rows.dim() != 2:
        raise ValueError(f"rows must be [T * k, d], not {tuple(rows.shape)}")
    n, d = rows.shape
    T = _routed("combine", routing, n)
    if y is None:
        y = rows.new_empty((T, d), dtype=torch.bfloat16)
    else:
        _need(y, "y", torch.bfloat16, T * d)
    _need(rows, "rows", torch.bfloat16, n * d)
    if base is not None:
        _need(base, "base", torch.bfloat16, T * d)
    _no_graph("combine", "its gradients are combine_grad's", rows=rows, base=base,
              topk_w=routing.topk_w if weighted else None)
    s = _launch_on("combine", rows=rows, base=base, y=y, inv_perm=routing.inv_perm)
    _check(_abi.lib().moe_combine(rows.data_ptr(), T, routing.k, d, C.addressof(routing.struct),
                                  0 if weighted else _abi.MOE_UNWEIGHTED, _ptr(base), y.data_ptr(), s),
           "moe_combine")
    return y


def combine_grad(dy: torch.Tensor, rows: torch.Tensor, routing: DeviceRouting,
                 d_rows: torch.Tensor | None = None, d_w: torch.Tensor | None = None, stream=None):
    """combine's gradients from dy [T, d] (bf16): (d_rows bf16 [T * k, d], d_w fp32 [T, k]).
    d_rows may be rows; base's gradient is dy.  d_w of a slot of weight 0 is 0 where its row
    makes it not finite."""
    if stream is not None:
        return _on_stream(combine_grad, locals())
    if dy.dim() != 2 or rows.dim() != 2 or dy.shape[1] != rows.shape[1]:
        raise ValueError(f"dy must be [T, d] and rows [T * k, d], not {tuple(dy.shape)}, "
                         f"{tuple(rows.shape)}")
    T, d = dy.shape
    n, k = rows.shape[0], routing.k
    _routed("combine_grad", routing, n, T)
    if d_rows is None:
        d_rows = torch.empty_like(rows)
    if d_w is None:
        d_w = dy.new_empty((T, k), dtype=torch.float32)
    _need(dy, "dy", torch.bfloat16, T * d)
    _need(rows, "rows", torch.bfloat16, n * d)
    _need(d_rows, "d_rows", torch.bfloat16, n * d)
    _need(d_w, "d_w", torch.float32, n)
    s = _launch_on("combine_grad", dy=dy, rows=rows, d_rows=d_rows, d_w=d_w,
                   inv_perm=routing.inv_perm)
    _check(_abi.lib().moe_combine_grad(_ptr(dy), _ptr(rows), T, k, d, C.addressof(routing.struct),
                                       _ptr(d_rows), _ptr(d_w), s), "moe_combine_grad")
    return d_rows, d_w


def penalize(logits: torch.Tensor, tokens: torch.Tensor | None = None,
             n_tokens: torch.Tensor | None = None, n_prompt: torch.Tensor | None = None,
             repetition=1.0, frequency=0.0, presence=0.0, bias_ids: torch.Tensor | None = None,
             bias: torch.Tensor | None = None, mask: torch.Tensor | None = None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Penalties, biases and a mask on rows of logits [B, V] (fp32), into out (which may be
    logits).  tokens: int32 [B, L], of which the first n_tokens [B] count (None: all) and
    those from n_prompt [B] on (None: all) are the answer; repetition (over all of them),
    frequency and presence (over the answer) are numbers for all rows or fp32 tensors [B];
    bias (fp32) is added at bias_ids (int32), both [B, n]; mask: int32 [B, ceil(V / 32)], bit
    v % 32 of word v / 32 is 1 where token v is allowed.  Ids outside 0 .. V - 1 (padding)
    are passed over."""
    if stream is not None:
        return _on_stream(penalize, locals())
    if logits.dim() != 2:
        raise ValueError(f"logits must be [B, V], not {tuple(logits.shape)}")
    B, V = logits.shape
    _need(logits, "logits", torch.float32, B * V)
    stride = n_bias = 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise ValueError(f"tokens must be [{B}, L], not {tuple(tokens.shape)}")
        _need(tokens, "tokens", torch.int32, 0)
        stride = tokens.shape[1]
    for name, t in (("n_tokens", n_tokens), ("n_prompt", n_prompt)):
        if t is not None:
            if tokens is None:
                raise ValueError(f"{name} needs tokens")
            _need(t, name, torch.int32, B)
    if tokens is not None and stride == 0:  # nothing to point at
        tokens = n_tokens = n_prompt = None
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias come together")
    if bias is not None:
        if bias_ids.dim() != 2 or bias_ids.shape[0] != B or bias.shape != bias_ids.shape:
            raise ValueError(f"bias_ids and bias must be [{B}, n], not {tuple(bias_ids.shape)}, "
                             f"{tuple(bias.shape)}")
        _need(bias_ids, "bias_ids", torch.int32, 0)
        _need(bias, "bias", torch.float32, 0)
        n_bias = bias.shape[1]
        if n_bias == 0:
            bias_ids = bias = None
    if mask is not None:
        if mask.dim() != 2 or tuple(mask.shape) != (B, (V + 31) >> 5):
            raise ValueError(f"mask must be [{B}, {(V + 31) >> 5}], not {tuple(mask.shape)}")
        _need(mask, "mask", torch.int32, 0)
    rep = freq = pres = None  # the parameters that are tensors
    if isinstance(repetition, torch.Tensor):
        _need(repetition, "repetition", torch.float32, B)
        rep, repetition = repetition, 0.0
    if isinstance(frequency, torch.Tensor):
        _need(frequency, "frequency", torch.float32, B)
        freq, frequency = frequency, 0.0
    if isinstance(presence, torch.Tensor):
        _need(presence, "presence", torch.float32, B)
        pres, presence = presence, 0.0
    if out is None:
        out = torch.empty_like(logits)
    else:
        _need(out, "out", torch.float32, B * V)
    s = _launch_on("penalize", logits=logits, out=out, tokens=tokens, n_tokens=n_tokens,
                   n_prompt=n_prompt, repetition=rep, frequency=freq, presence=pres,
                   bias_ids=bias_ids, bias=bias, mask=mask)
    # (the struct's bytes: building a ctypes structure of 14 fields costs 2 us)
    p = _abi.PENALTIES(0 if tokens is None else tokens.data_ptr(),
                       0 if n_tokens is None else n_tokens.data_ptr(),
                       0 if n_prompt is None else n_prompt.data_ptr(),
                       0 if rep is None else rep.data_ptr(), 0 if freq is None else freq.data_ptr(),
                       0 if pres is None else pres.data_ptr(),
                       0 if bias_ids is None else bias_ids.data_ptr(),
                       0 if bias is None else bias.data_ptr(), 0 if mask is None else mask.data_ptr(),
                       stride, n_bias, repetition, frequency, presence)
    _check(_abi.lib().moe_penalize(logits.data_ptr(), B, V, p, out.data_ptr(), s), "moe_penalize")
    return out


def library_path() -> str:
    return _abi.LIB_PATH
