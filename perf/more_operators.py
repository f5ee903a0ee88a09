"""Measured calls of the 8-bit expert products and the operators next to them.

Four operators, each with its plain form (elementary torch operations) and the
call a user makes of the library:

  linear    y = W x in e4m3, with one fp32 scale per token and 128 columns of x and
            one per 128 x 128 block of W; fp32 or bf16 out, or gated: W holds a
            gate and an up matrix and silu(gate) * up goes out in e4m3 with a
            scale per token and 128 columns
  experts   the same products over expert-sorted rows, a matrix per expert
  sort      token rows into expert order (bf16, or e4m3 with scales), expert rows
            back to their tokens with the routing weights, and the gradients
  penalize  repetition, frequency and presence penalties, sparse biases and a
            grammar's bit mask on rows of logits

`own` chooses between the two forms.  Sizes are those of the repository's
workloads (d = 2048, experts of 512, 256 experts, top-8, chunks of 512 to 32768
tokens, heads of 3000 and 248320 rows, hidden sizes up to 8192) and odd ones
around them.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128       # columns (and weight rows) that share a scale
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _linear(name, T, N, K, out="bfloat16"):
    """N rows of weights; out "gated": a gate and an up matrix of N / 2 rows each."""
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "out": out}


def _experts(name, T, E, k, N, K, out="bfloat16", skew=0.3):
    return {"name": name, "op": "experts", "T": T, "E": E, "k": k, "N": N, "K": K, "out": out,
            "skew": skew}


def _sort(name, kind, T, E, k, d, skew=0.3):
    return {"name": name, "op": "sort", "kind": kind, "T": T, "E": E, "k": k, "d": d, "skew": skew}


def _penalize(name, B, V, history, biases=0, masked=0.0):
    return {"name": name, "op": "penalize", "B": B, "V": V, "history": history, "biases": biases,
            "masked": masked}


def listed():
    return [
        # one token through a projection of the hidden size: latency
        _linear("linear_token", 1, 2048, 2048),
        # an odd number of rows and tokens, a last block of half the columns, fp32 logits
        _linear("linear_odd", 1001, 3001, 2112, "float32"),
        # a long prompt through a projection of the largest hidden size: matrix cores
        _linear("linear_chunk", 8192, 8192, 8192),
        # eight decoded tokens through their experts' gate and up matrices: weight stream
        _experts("experts_decode", 8, 256, 8, 1024, 2048, "gated"),
        # the headline prefill chunk through gate and up: every expert's weights once
        _experts("experts_gate_up", 2048, 256, 8, 1024, 2048, "gated"),
        # a longer, skewed chunk through the down matrices
        _experts("experts_down", 4096, 256, 8, 2048, 512, skew=0.8),
        # a prefill chunk into expert order in 8 bits
        _sort("dispatch_e4m3", "dispatch_e4m3", 2048, 256, 8, 2048),
        # one token's expert rows back to it: latency
        _sort("combine_token", "combine", 1, 256, 8, 2048),
        # a training batch's way back: gradients of the expert rows and of the weights
        _sort("combine_grad", "combine_grad", 8192, 256, 8, 2048),
        # one sequence with penalties on a long answer: latency
        _penalize("penalize_one", 1, 248320, 2000),
        # a serving batch of which every row has a grammar's mask and some biases
        _penalize("penalize_batch", 64, 248320, 4000, 100, 0.9),
        # an odd batch on a small head
        _penalize("penalize_small", 37, 3001, 500, 20, 0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "experts", "sort", "penalize"])
    out = rng.choice(["bfloat16", "float32", "gated"])
    if op == "linear":
        K = 64 * _log_int(rng, 1, 128)
        N = 128 * _log_int(rng, 1, 64) if out == "gated" else _log_int(rng, 16, 30000)
        return _linear("", _log_int(rng, 1, min(8192, (1 << 39) // (N * K))), N, K, out)
    E = rng.choice([8, 32, 256, rng.randint(2, 256)])
    k = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.3, 0.8])
    if op == "experts":
        K = 64 * _log_int(rng, 1, 64)
        rows = min(8192, 536870912 // (E * K))
        N = 128 * _log_int(rng, 1, rows // 128) if out == "gated" else _log_int(rng, 16, rows)
        return _experts("", _log_int(rng, 1, min(4096, (1 << 34) // (k * N * K) + 1)), E, k, N, K,
                        out, skew)
    if op == "sort":
        d = 64 * _log_int(rng, 1, 128)
        T = _log_int(rng, 1, min(32768, 134217728 // (k * d)))
        return _sort("", rng.choice(["dispatch", "dispatch_e4m3", "combine", "combine_plain",
                                     "combine_grad"]), T, E, k, d, skew)
    B = _log_int(rng, 1, 64)
    return _penalize("", B, _log_int(rng, 1000, 248320), _log_int(rng, 1, 32768),
                     rng.choice([0, 0, 5, 300]), rng.choice([0.0, 0.0, 0.5, 0.99]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _up(n, m):
    return -(-n // m)


def _codes(v, scale):
    return torch.where(scale > 0, v / scale, 0.0).clamp(-E4M3_MAX, E4M3_MAX).to(
        torch.float8_e4m3fn)


def _quant_rows(x):
    """e4m3 codes and a scale per row and 128 columns."""
    T, K = x.shape
    g = torch.nn.functional.pad(x.float(), (0, _up(K, BLOCK) * BLOCK - K)).view(T, -1, BLOCK)
    scale = g.abs().amax(2) / E4M3_MAX
    codes = _codes(g, scale.unsqueeze(2)).view(T, -1)
    return codes[:, :K].contiguous(), scale


def _quant_blocks(w):
    """e4m3 codes of [M, N, K] and a scale per 128 x 128 block of each matrix."""
    M, N, K = w.shape
    nb, kb = _up(N, BLOCK), _up(K, BLOCK)
    if N % BLOCK or K % BLOCK:
        w = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N))
    g = w.view(M, nb, BLOCK, kb, BLOCK)
    scale = torch.maximum(g.amax((2, 4)), -g.amin((2, 4))) / E4M3_MAX
    codes = g.div_(scale[:, :, None, :, None].clamp(min=1e-30)).to(torch.float8_e4m3fn)
    return codes.view(M, nb * BLOCK, kb * BLOCK)[:, :N, :K].contiguous(), scale


def _routing(case, rn):
    """Selections and weights of T tokens, and the expert-sorted order."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = rn(T, E) + case["skew"] * rn(E)
    top, idx = logits.sort(dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    w = torch.softmax(top, 1)
    perm = idx.reshape(-1).sort(stable=True).indices
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device=perm.device))
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    return {"logits": logits, "idx": idx, "w": w.contiguous(), "perm": perm, "inv": inv,
            "counts": counts, "most": int(counts.max())}


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    rn = lambda *shape: torch.randn(shape, generator=g, device=dev)            # noqa: E731
    ru = lambda *shape: torch.rand(shape, generator=g, device=dev)             # noqa: E731
    ri = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device=dev)  # noqa: E731
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("linear", "experts"):
        N, K = case["N"], case["K"]
        rows = case["T"]
        if op == "experts":
            s["routing"] = _routing(case, rn)
            rows *= case["k"]
        # normalised rows with some columns larger than the rest, as hidden states have
        s["x"], s["x_scale"] = _quant_rows(rn(rows, K) * (1.0 + 9.0 * (ru(K) < 0.01)))
        E = case["E"] if op == "experts" else 1
        parts = 2 if case["out"] == "gated" else 1
        w = rn(E * parts, N // parts, K) * K ** -0.5
        w8, scale = _quant_blocks(w)
        lead = ((E,) if op == "experts" else ()) + ((2,) if parts == 2 else ())
        s["w"] = w8.view(*lead, *w8.shape[1:])
        s["w_scale"] = scale.view(*lead, *scale.shape[1:])
    elif op == "sort":
        T, k, d = case["T"], case["k"], case["d"]
        s["routing"] = _routing(case, rn)
        if case["kind"].startswith("dispatch"):
            s["x"] = rn(T, d).to(torch.bfloat16)
        else:
            s["rows"] = (0.3 * rn(T * k, d)).to(torch.bfloat16)
            if case["kind"] == "combine":  # the shared expert's output
                s["base"] = (0.3 * rn(T, d)).to(torch.bfloat16)
            if case["kind"] == "combine_grad":
                s["dy"] = (1e-3 * rn(T, d)).to(torch.bfloat16)
    else:
        B, V, H = case["B"], case["V"], case["history"]
        logits = 2.0 * rn(B, V)
        # some tokens come often, and those that came are likely to come again
        tokens = (V * ru(B, H) ** 6).long().clamp(max=V - 1)
        s["logits"] = logits.scatter_add_(1, tokens, torch.full_like(tokens, 0.5, dtype=torch.float32))
        n = ri(H + 1, B)
        n[0] = H
        s["n_tokens"] = n.int()
        s["n_prompt"] = (n * ru(B)).int()
        live = torch.arange(H, device=dev) < n[:, None]
        s["tokens"] = torch.where(live, tokens, -1).int()
        s["repetition"] = 1.0 + 0.3 * ru(B)
        s["frequency"] = 0.5 * ru(B)
        s["presence"] = ru(B) - 0.3
        s["bias_ids"] = s["bias"] = s["mask"] = None
        if case["biases"]:
            s["bias_ids"] = ri(V, B, case["biases"]).int()
            s["bias"] = 5.0 * rn(B, case["biases"])
        if case["masked"]:
            bits = ru(B, _up(V, 32) * 32) >= case["masked"]
            if B > 1:
                bits[B - 1] = False  # a grammar that has come to its end
            sh = torch.arange(32, device=dev)
            words = (bits.view(B, -1, 32).long() << sh).sum(2)
            s["mask"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "routing" in s:  # the routing arrays that a serving program keeps
        import q4_routed_expert_amd as q4
        dev = torch.device("cuda")
        E, k = case["E"], case["k"]
        t = {m + "_q": torch.zeros(E * 64 * 8, dtype=torch.int32, device=dev) for m in q4.MATS}
        t |= {m + z: torch.zeros(E * 64, dtype=torch.int16, device=dev) for m in q4.MATS
              for z in ("_s", "_b")}
        t["w_router"] = torch.zeros(64 * E, device=dev)
        r = q4.DeviceRouting(case["T"], E, k, dev)
        r.logits.copy_(s["routing"]["logits"])
        x = torch.zeros((case["T"], 64), dtype=torch.bfloat16, device=dev)
        q4.route(q4.DeviceLayer(64, 64, E, k, t), x, routing=r, logits_in=True)
        r.topk_w.copy_(s["routing"]["w"])
        s["own_routing"] = r
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _expand_rows(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]


def _expand_blocks(codes, scale):
    N, K = codes.shape[-2:]
    s = scale.repeat_interleave(BLOCK, -1)[..., :K].repeat_interleave(BLOCK, -2)[..., :N, :]
    return codes.float() * s


def _gate(y):
    """silu(first half) * second half in 8 bits."""
    g, u = y.chunk(2, 1)
    codes, scale = _quant_rows(g / (1.0 + torch.exp(-g)) * u)
    return {"y8": codes, "scale": scale}


def _finish(y, out):
    return _gate(y) if out == "gated" else y.to(getattr(torch, out))


def _plain_linear(s):
    w = _expand_blocks(s["w"], s["w_scale"])
    y = _expand_rows(s["x"], s["x_scale"]) @ w.view(-1, w.shape[-1]).t()
    return _finish(y, s["case"]["out"])


def _plain_experts(s):
    r, c = s["routing"], s["case"]
    E, N, K, most = c["E"], c["N"], c["K"], s["routing"]["most"]
    x = _expand_rows(s["x"], s["x_scale"])
    w = _expand_blocks(s["w"], s["w_scale"]).view(E, N, K)
    # every expert's rows padded to the most that one has
    first = torch.cumsum(r["counts"], 0) - r["counts"]
    at = torch.arange(most, device=x.device)
    pick = (first[:, None] + at).clamp(max=x.shape[0] - 1)
    y = torch.bmm(w, x[pick].transpose(1, 2).contiguous())                  # [E, N, most]
    expert = torch.repeat_interleave(r["counts"], output_size=x.shape[0])
    row = torch.arange(x.shape[0], device=x.device)
    return _finish(y.transpose(1, 2)[expert, row - first[expert]], c["out"])


def _plain_sort(s):
    r, c = s["routing"], s["case"]
    T, k, kind = c["T"], c["k"], c["kind"]
    if kind.startswith("dispatch"):
        token = torch.div(r["perm"], k, rounding_mode="floor")
        if kind == "dispatch":
            return s["x"][token]
        codes, scale = _quant_rows(s["x"])
        return {"rows": codes.view(torch.uint8)[token].view(torch.float8_e4m3fn),
                "scale": scale[token]}
    if kind == "combine_grad":
        dy, rows = s["dy"].float(), s["rows"].float()[r["inv"]].view(T, k, -1)
        d_rows = (r["w"].unsqueeze(2) * dy.unsqueeze(1)).to(torch.bfloat16)
        return {"d_rows": d_rows.view(T * k, -1)[r["perm"]],
                "d_w": (rows * dy.unsqueeze(1)).sum(2)}
    rows = s["rows"].float()[r["inv"]].view(T, k, -1)
    y = rows.sum(1) if kind == "combine_plain" else (rows * r["w"].unsqueeze(2)).sum(1)
    if "base" in s:
        y = y + s["base"].float()
    return y.to(torch.bfloat16)


def _plain_penalize(s):
    l, V = s["logits"], s["logits"].shape[1]
    at = torch.arange(s["tokens"].shape[1], device=l.device)
    live = at < s["n_tokens"][:, None]
    answer = live & (at >= s["n_prompt"][:, None])
    ids = torch.where(live, s["tokens"], 0).long()
    zero = torch.zeros_like(l)
    seen = zero.scatter_add(1, ids, live.float()) > 0
    count = zero.scatter_add(1, ids, answer.float())
    rep = s["repetition"][:, None]
    y = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
    y = y - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"] is not None:
        y = (y.double().scatter_add_(1, s["bias_ids"].long(), s["bias"].double())).float()
    if s["mask"] is not None:
        v = torch.arange(V, device=l.device)
        allowed = (s["mask"][:, v // 32] >> (v % 32)) & 1
        y = torch.where(allowed > 0, y, -math.inf)
    return y


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_product(s, call, *routing):
    out = s["case"]["out"]
    if out == "gated":
        y8, scale = call(s["w"], s["w_scale"], s["x"], s["x_scale"], *routing, gated=True)
        return {"y8": y8, "scale": scale}
    return call(s["w"], s["w_scale"], s["x"], s["x_scale"], *routing,
                out_dtype=getattr(torch, out))


def _own_linear(s):
    import q4_routed_expert_amd as q4
    return _own_product(s, q4.linear_e4m3)


def _own_experts(s):
    import q4_routed_expert_amd as q4
    return _own_product(s, q4.experts_e4m3, s["own_routing"])


def _own_sort(s):
    import q4_routed_expert_amd as q4
    r, kind = s["own_routing"], s["case"]["kind"]
    if kind == "dispatch":
        return q4.dispatch(s["x"], r)[0]
    if kind == "dispatch_e4m3":
        rows, scale = q4.dispatch(s["x"], r, e4m3=True)
        return {"rows": rows, "scale": scale}
    if kind == "combine_grad":
        d_rows, d_w = q4.combine_grad(s["dy"], s["rows"], r)
        return {"d_rows": d_rows, "d_w": d_w}
    return q4.combine(s["rows"], r, weighted=kind == "combine", base=s.get("base"))


def _own_penalize(s):
    import q4_routed_expert_amd as q4
    return q4.penalize(s["logits"], tokens=s["tokens"], n_tokens=s["n_tokens"],
                       n_prompt=s["n_prompt"], repetition=s["repetition"],
                       frequency=s["frequency"], presence=s["presence"],
                       bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "experts": _own_experts, "sort": _own_sort,
                "penalize": _own_penalize}[op](state)
    return {"linear": _plain_linear, "experts": _plain_experts, "sort": _plain_sort,
            "penalize": _plain_penalize}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("linear", "experts"):
        N, K, rows, mats = case["N"], case["K"], case["T"], 1.0
        if op == "experts":  # the experts that T tokens reach when all are equally likely
            mats = case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** rows)
            rows *= case["k"]
        out = {"bfloat16": 2 * N, "float32": 4 * N, "gated": N // 2 + 4 * _up(N // 2, BLOCK)}
        w = N * K + 4 * _up(N, BLOCK) * _up(K, BLOCK)
        return {"bytes": int(mats * w) + rows * (K + 4 * _up(K, BLOCK) + out[case["out"]]),
                "flops": 2 * rows * N * K}
    if op == "sort":
        T, k, d, kind = case["T"], case["k"], case["d"], case["kind"]
        if kind.startswith("dispatch"):
            size = 2 * d if kind == "dispatch" else d + 4 * _up(d, BLOCK)
            return {"bytes": 2 * T * d + T * k * (4 + size), "flops": 0}
        if kind == "combine_grad":
            return {"bytes": 2 * T * d + T * k * (4 * d + 12), "flops": 3 * T * k * d}
        return {"bytes": (4 if kind == "combine" else 2) * T * d + T * k * (2 * d + 8),
                "flops": 2 * T * k * d}
    B, V = case["B"], case["V"]
    mask = 4 * B * _up(V, 32) if case["masked"] else 0
    return {"bytes": 8 * B * V + mask + 4 * B * case["history"] + 8 * B * case["biases"],
            "flops": B * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _wide(codes, scale, rows):
    """The values in 64 bits of a matrix of codes with a scale per `rows` x 128 block."""
    n = torch.arange(codes.shape[0], device=codes.device) // rows
    kk = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.float().double() * scale.double()[n][:, kk]


def _exact_product(x, w):
    """x [rows, K] in 64 bits times the transposed matrix or matrices of (codes, scale)."""
    return torch.cat([torch.mm(x, _wide(c, sc, BLOCK).t().contiguous()) for c, sc in w], 1)


def _exact_out(y, out):
    if out != "gated":
        return y
    g, u = y[:, :y.shape[1] // 2], y[:, y.shape[1] // 2:]
    h = g * torch.sigmoid(g) * u
    scale = torch.stack([p.abs().max(1).values for p in h.split(BLOCK, 1)], 1) / E4M3_MAX
    kk = torch.arange(h.shape[1], device=h.device) // BLOCK
    return {"y8": h / scale[:, kk].clamp(min=1e-300), "scale": scale}


def _exact_linear(s):
    w = zip(s["w"], s["w_scale"]) if s["w"].dim() == 3 else [(s["w"], s["w_scale"])]
    return _exact_out(_exact_product(_wide(s["x"], s["x_scale"], 1), w), s["case"]["out"])


def _exact_experts(s):
    x, parts, row = _wide(s["x"], s["x_scale"], 1), [], 0
    for e, n in enumerate(s["routing"]["counts"].tolist()):
        if n:
            w = s["w"][e], s["w_scale"][e]
            w = zip(*w) if w[0].dim() == 3 else [w]
            parts.append(_exact_product(x[row:row + n], w))
        row += n
    return _exact_out(torch.cat(parts), s["case"]["out"])


def _exact_sort(s):
    c, r = s["case"], s["routing"]
    T, k, d, kind = c["T"], c["k"], c["d"], c["kind"]
    order = torch.from_numpy(np.argsort(r["idx"].cpu().numpy().reshape(-1), kind="stable"))
    order = order.to(r["idx"].device)
    if kind == "dispatch":
        return s["x"].double()[order // k]
    if kind == "dispatch_e4m3":
        x = s["x"].double()
        scale = torch.stack([p.abs().max(1).values for p in x.split(BLOCK, 1)], 1) / E4M3_MAX
        kk = torch.arange(d, device=x.device) // BLOCK
        return {"rows": (x / scale[:, kk].clamp(min=1e-300))[order // k],
                "scale": scale[order // k]}
    w = r["w"].double().reshape(-1)[order]
    if kind == "combine_grad":
        dy = s["dy"].double()[order // k]
        d_w = torch.empty(T * k, dtype=torch.float64, device=dy.device)
        d_w[order] = (s["rows"].double() * dy).sum(1)
        return {"d_rows": w[:, None] * dy, "d_w": d_w.view(T, k)}
    y = torch.zeros((T, d), dtype=torch.float64, device=w.device)
    y.index_add_(0, order // k, s["rows"].double() * (w[:, None] if kind == "combine" else 1.0))
    return y + s["base"].double() if "base" in s else y


def _exact_penalize(s):
    host = {n: v.cpu().numpy() for n, v in s.items() if isinstance(v, torch.Tensor)}
    y = host["logits"].astype(np.float64)
    V = y.shape[1]
    for b, row in enumerate(y):
        n, p = int(host["n_tokens"][b]), int(host["n_prompt"][b])
        seen = np.unique(host["tokens"][b, :n])
        row[seen] *= np.where(row[seen] > 0, 1.0 / float(host["repetition"][b]),
                              float(host["repetition"][b]))
        ids, count = np.unique(host["tokens"][b, p:n], return_counts=True)
        row[ids] -= float(host["frequency"][b]) * count + float(host["presence"][b])
        if "bias" in host:
            np.add.at(row, host["bias_ids"][b], host["bias"][b].astype(np.float64))
        if "mask" in host:
            bits = np.unpackbits(host["mask"][b].view(np.uint8), bitorder="little")[:V]
            row[bits == 0] = -np.inf
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    return {"linear": _exact_linear, "experts": _exact_experts, "sort": _exact_sort,
            "penalize": _exact_penalize}[case["op"]](s)
