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
    token, prob, _ = sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)
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


# The current stream's handle without building a stream object (2.5 us of a call).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch_on(where: str, **tensors) -> int:
    """The current stream's handle for a call whose tensors are `tensors` (None: absent).
    All of them have to be on one GPU, and that GPU has to be the current one, because
    the library launches on the current device."""
    dev = -1
    for name, t in tensors.items():
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{name} must be on the GPU")
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError(f"{where}: {name} is on cuda:{d}, other arguments on cuda:{dev}")
    if dev != torch.cuda.current_device():
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


def add_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
             eps: float = 1e-6, plus_one: bool = False, residual_out: torch.Tensor | None = None,
             y: torch.Tensor | None = None, e4m3: bool = False, y8: torch.Tensor | None = None,
             y8_scale: torch.Tensor | None = None, stream=None):
    """Residual addition and RMS norm of the rows of x [T, d] (bf16): (y, y8, y8_scale).

    residual: bf16 or fp32 [T, d]; x + residual goes to residual_out (which may be
    residual itself; None: not stored).  plus_one: the weight used is weight + 1.
    y (bf16) is written when given, and by default when no 8-bit output is asked
    for; e4m3=True (or y8 and y8_scale given) asks for e4m3 codes [T, d] with one
    fp32 scale per 64 columns [T, d / 64]."""
    if stream is not None:
        return _on_stream(add_norm, locals())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], not {tuple(x.shape)}")
    T, d = x.shape
    flags = _abi.MOE_NORM_PLUS_ONE if plus_one else 0
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
            y8_scale = x.new_empty((T, d // 64), dtype=torch.float32)
        _need(y8, "y8", torch.float8_e4m3fn, T * d)
        _need(y8_scale, "y8_scale", torch.float32, T * (d // 64))
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


def library_path() -> str:
    return _abi.LIB_PATH
