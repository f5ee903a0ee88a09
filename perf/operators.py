"""Measured calls of the operators around the routed-MoE layer.

Four operators, each with its plain form (elementary torch operations) and the
call a user makes of the library:

  route   expert routing from fp32 router logits: softmax or sigmoid scores, a
          per-expert bias that steers the selection only, expert groups, top-k,
          renormalised and scaled weights, and the expert-sorted order that the
          grouped products walk
  linear  y = W x for 1 .. 64 rows of bf16 activations against one group-64
          affine 4-bit matrix (the experts' weight format)
  sample  one token per row of logits, with temperature, top-k, top-p and min-p,
          from a given uniform number per row, and that token's probability
  norm    residual addition and root-mean-square norm, with a bf16 output or an
          e4m3 output with one scale per 64 columns

`own` chooses between the two forms.  Sizes are those of the repository's
workloads (d = 2048, 256 experts, top-8, chunks of 512 to 32768 tokens, output
heads of 3000 and 248320 rows) and odd ones around them.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64        # columns per quantisation group (weights, and the 8-bit output)
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(name, T, E, k, score="sigmoid", groups=1, keep=1, group_top=1, balance=True,
           renorm=True, scale=1.0):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
            "keep": keep, "group_top": group_top, "balance": balance, "renorm": renorm,
            "scale": scale}


def _linear(name, T, N, K, out="float32"):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "out": out}


def _sample(name, B, V, temperature=0.8, top_k=0, top_p=1.0, min_p=0.0, spread=2.0, coarse=False,
            masked=0.0):
    return {"name": name, "op": "sample", "B": B, "V": V, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "spread": spread, "coarse": coarse,
            "masked": masked}


def _norm(name, T, d, residual="bfloat16", out="bfloat16", plus_one=False):
    return {"name": name, "op": "norm", "T": T, "d": d, "residual": residual, "out": out,
            "plus_one": plus_one}


def listed():
    return [
        # one decoded token's routing, with groups: pure latency
        _route("route_token", 1, 256, 8, groups=8, keep=4, group_top=2, scale=2.5),
        # the prefill chunk of the headline workload, softmax scores with a balance bias
        _route("route_chunk", 2048, 256, 8, score="softmax"),
        # the longest chunk the library takes, sigmoid scores and groups
        _route("route_long", 32768, 256, 8, groups=8, keep=4, group_top=2, scale=2.5),
        # one token through a projection of the hidden size: latency
        _linear("linear_token", 1, 2048, 2048, "bfloat16"),
        # the output head for a few decoded or drafted tokens: the weight stream
        _linear("linear_head", 8, 248320, 2048),
        # a full batch through an odd number of rows of the largest hidden size
        _linear("linear_batch", 64, 30011, 8192, "bfloat16"),
        # one sequence's next token with every filter on: latency
        _sample("sample_one", 1, 248320, top_k=50, top_p=0.95, min_p=0.02),
        # a serving batch with top-p alone, logits that were computed in bf16 (many ties)
        _sample("sample_batch", 64, 248320, temperature=1.0, top_p=0.9, coarse=True),
        # an odd batch on a small head, temperature alone
        _sample("sample_small", 37, 3001, temperature=1.3),
        # one token between two layers: latency
        _norm("norm_token", 1, 2048),
        # a prefill chunk whose output goes on in 8 bits
        _norm("norm_chunk_e4m3", 2048, 2048, out="e4m3", plus_one=True),
        # the longest chunk, an fp32 residual stream
        _norm("norm_long", 32768, 2048, residual="float32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "linear", "sample", "norm"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        per = rng.randint(2, 256 // groups)
        E = groups * per
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(8, keep * per))
        return {**_route("", _log_int(rng, 1, 32768), E, k, rng.choice(["softmax", "sigmoid"]),
                         groups, keep, rng.choice([1, 2]), rng.random() < 0.7, rng.random() < 0.7,
                         rng.choice([1.0, 2.5]))}
    if op == "linear":
        K = GROUP * _log_int(rng, 1, 128)
        most = min(248320, 508559360 // K)  # no more weights than the output head's
        return _linear("", _log_int(rng, 1, 64), _log_int(rng, 16, most), K,
                       rng.choice(["float32", "bfloat16"]))
    if op == "sample":
        B = _log_int(rng, 1, 64)
        return _sample("", B, _log_int(rng, 1000, 248320), rng.choice([0.0, 0.5, 0.8, 1.0, 1.5]),
                       rng.choice([0, 0, 1, 20, 50, 1000]), rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]),
                       rng.choice([0.0, 0.0, 0.02, 0.1]), rng.uniform(1.0, 3.0),
                       rng.random() < 0.5, rng.choice([0.0, 0.0, 0.5, 0.99]))
    d = GROUP * _log_int(rng, 1, 128)
    T = _log_int(rng, 1, min(32768, 67108864 // d))
    return _norm("", T, d, rng.choice(["none", "bfloat16", "float32"]),
                 rng.choice(["bfloat16", "e4m3"]), rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    rn = lambda *shape: torch.randn(shape, generator=g, device=dev)            # noqa: E731
    ru = lambda *shape: torch.rand(shape, generator=g, device=dev)             # noqa: E731
    op = case["op"]
    s = {"case": dict(case)}
    if op == "route":
        # x ~ N(0, 1) against W_r ~ N(0, 1/d) gives logits ~ N(0, 1)
        s["logits"] = rn(case["T"], case["E"])
        s["balance"] = 0.1 * rn(case["E"]) if case["balance"] else None
    elif op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = rn(T, K).to(torch.bfloat16)
        s["q"] = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device=dev,
                               dtype=torch.int32)
        scale = (0.005 + 0.010 * ru(N, K // GROUP)).to(torch.bfloat16)
        s["scale"] = scale
        s["bias"] = (-8.0 * scale.float() + 0.002 * (ru(N, K // GROUP) - 0.5)).to(torch.bfloat16)
    elif op == "sample":
        B, V = case["B"], case["V"]
        logits = case["spread"] * rn(B, V)
        # a few likely tokens above the bulk, as a trained head gives
        top = torch.randint(0, V, (B, 12), generator=g, device=dev)
        logits.scatter_add_(1, top, 4.0 * case["spread"] + 3.0 * rn(B, 12))
        logits = logits.to(torch.bfloat16).float() if case["coarse"] else logits
        if case["masked"]:  # tokens that a grammar rules out
            logits.masked_fill_(ru(B, V) < case["masked"], -math.inf)
        s["logits"] = logits
        s["u"] = ru(B)
        full = lambda v, t: torch.full((B,), v, dtype=t, device=dev)           # noqa: E731
        s["temperature"] = full(case["temperature"], torch.float32)
        s["top_k"] = full(case["top_k"], torch.int32)
        s["top_p"] = full(case["top_p"], torch.float32)
        s["min_p"] = full(case["min_p"], torch.float32)
    else:
        T, d = case["T"], case["d"]
        s["x"] = rn(T, d).to(torch.bfloat16)
        s["weight"] = ((0.0 if case["plus_one"] else 1.0) + 0.2 * rn(d)).to(torch.bfloat16)
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = (4.0 * rn(T, d)).to(getattr(torch, case["residual"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the buffers and handles that a serving program keeps
        import q4_routed_expert_amd as q4
        dev = torch.device("cuda")
        if case["op"] == "route":
            E, k = case["E"], case["k"]
            t = {m + "_q": torch.zeros(E * 64 * 8, dtype=torch.int32, device=dev) for m in q4.MATS}
            t |= {m + z: torch.zeros(E * 64, dtype=torch.int16, device=dev) for m in q4.MATS
                  for z in ("_s", "_b")}
            t["w_router"] = torch.zeros(64 * E, device=dev)
            s["layer"] = q4.DeviceLayer(64, 64, E, k, t)
            s["routing"] = q4.DeviceRouting(case["T"], E, k, dev)
            s["routing"].logits.copy_(s["logits"])
            s["spec"] = q4.RouterSpec(score=case["score"], n_groups=case["groups"],
                                      top_groups=case["keep"], group_top=case["group_top"],
                                      renorm=case["renorm"], scale=case["scale"],
                                      balance=s["balance"])
        elif case["op"] == "sample":
            s["ws"] = q4.sample_workspace(case["B"], case["V"], dev)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _tiles(counts, offsets, rows, cap):
    """(expert, first sorted row) of every `rows`-row tile, experts ascending, and their number."""
    n = torch.div(counts + rows - 1, rows, rounding_mode="floor")
    end = torch.cumsum(n, 0)
    j = torch.arange(cap, device=counts.device)
    e = torch.searchsorted(end, j, right=True).clamp(max=counts.numel() - 1)
    row = offsets[e] + rows * (j - (end - n)[e])
    live = j < end[-1]
    tiles = torch.stack([torch.where(live, e, 0), torch.where(live, row, 0)], 1)
    return tiles.to(torch.int32), end[-1:].to(torch.int32)


def _plain_route(s):
    c, E, k = s["case"], s["case"]["E"], s["case"]["k"]
    l = s["logits"].double()  # scores next to a selection border need more than 32 bits
    T = l.shape[0]
    if c["score"] == "softmax":
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    sel = score if s["balance"] is None else score + s["balance"].double()
    if c["groups"] > 1:
        G = c["groups"]
        best = sel.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        live = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        sel = torch.where(live.repeat_interleave(E // G, 1), sel, -math.inf)
    idx = sel.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * c["scale"]).float()
    flat = idx.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=l.device).scatter_add_(
        0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    perm = flat.sort(stable=True).indices
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device=l.device))
    cap = lambda rows: T * k // rows + min(E, T * k)                           # noqa: E731
    bm, nb = _tiles(counts, offsets[:-1], 32, cap(32))
    tm, nt = _tiles(counts, offsets[:-1], 128, cap(128))
    i32 = lambda t: t.to(torch.int32)                                          # noqa: E731
    return {"idx": i32(idx), "w": w, "counts": i32(counts), "offsets": i32(offsets),
            "perm": i32(perm), "inv_perm": i32(inv), "block_map": bm, "n_blocks": nb,
            "tile_map": tm, "n_tiles": nt}


def _plain_linear(s):
    q, scale, bias, x = s["q"], s["scale"], s["bias"], s["x"]
    N, words = q.shape
    shifts = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    step = max(1, (1 << 28) // (8 * words))  # a bounded number of expanded weights at a time
    out = []
    for n in range(0, N, step):
        codes = torch.bitwise_and(q[n:n + step].unsqueeze(2) >> shifts, 15)
        codes = codes.view(-1, words // 8, GROUP).float()
        w = codes * scale[n:n + step].float().unsqueeze(2) + bias[n:n + step].float().unsqueeze(2)
        w = w.to(torch.bfloat16).float().view(-1, 8 * words)  # a weight is the bf16 value
        out.append(x.float() @ w.t())
    return torch.cat(out, 1).to(getattr(torch, s["case"]["out"]))


def _plain_sample(s):
    # cumulated weights next to a border need more than 32 bits
    l = torch.nan_to_num(s["logits"].double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    V = l.shape[1]
    temp = s["temperature"].double().unsqueeze(1)
    greedy = temp <= 0
    w = torch.exp((l - l.amax(1, keepdim=True)) / torch.where(greedy, 1.0, temp))
    order = l.sort(dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device=l.device).unsqueeze(0)
    k = s["top_k"].long().unsqueeze(1)
    k = torch.where((k <= 0) | (k > V), V, k)
    k = torch.where(greedy, 1, k)
    keep = rank < k
    mass = torch.cumsum(torch.where(keep, ws, 0.0), 1)
    p = s["top_p"].double().unsqueeze(1)
    keep &= (mass - ws < p * mass[:, -1:]) | (p >= 1) | (rank == 0)
    keep &= ws >= s["min_p"].double().unsqueeze(1)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    cum = torch.cumsum(torch.where(kept, w, 0.0), 1)
    target = s["u"].double().unsqueeze(1) * cum[:, -1:]
    token = ((cum > target) & kept).to(torch.int8).argmax(1, keepdim=True)
    prob = w.gather(1, token) / cum[:, -1:]  # in the distribution that it was drawn from
    return {"token": token.view(-1).to(torch.int32), "prob": prob.view(-1).float()}


def _plain_norm(s):
    c = s["case"]
    v = s["x"].float()
    out = {}
    if s["residual"] is not None:
        r = (v + s["residual"].float()).to(s["residual"].dtype)
        out["residual"] = r
        v = r.float()
    w = s["weight"].float() + (1.0 if c["plus_one"] else 0.0)
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w
    if c["out"] == "bfloat16":
        out["y"] = y.to(torch.bfloat16)
        return out
    yg = y.view(y.shape[0], -1, GROUP)
    scale = yg.abs().amax(2) / E4M3_MAX
    inv = torch.where(scale > 0, 1.0 / scale, 0.0)
    out["y8"] = (yg * inv.unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(
        torch.float8_e4m3fn)
    out["scale"] = scale
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_route(s):
    import q4_routed_expert_amd as q4
    r = q4.route_scored(s["layer"], None, s["spec"], s["routing"], logits_in=True)
    return {"idx": r.topk_idx, "w": r.topk_w, "counts": r.counts, "offsets": r.offsets,
            "perm": r.perm, "inv_perm": r.inv_perm, "block_map": r.block_map,
            "n_blocks": r.n_blocks, "tile_map": r.tile_map, "n_tiles": r.n_tiles}


def _own_linear(s):
    import q4_routed_expert_amd as q4
    return q4.linear(s["q"], s["scale"], s["bias"], s["x"],
                     out_dtype=getattr(torch, s["case"]["out"]))


def _own_sample(s):
    import q4_routed_expert_amd as q4
    token, prob, _ = q4.sample(s["logits"], s["u"], temperature=s["temperature"],
                               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], ws=s["ws"])
    return {"token": token, "prob": prob}


def _own_norm(s):
    import q4_routed_expert_amd as q4
    c, out = s["case"], {}
    r = s["residual"]
    if r is not None:
        out["residual"] = torch.empty_like(r)
    y, y8, scale = q4.add_norm(s["x"], s["weight"], r, eps=1e-6, plus_one=c["plus_one"],
                               e4m3=c["out"] == "e4m3", residual_out=out.get("residual"))
    if c["out"] == "bfloat16":
        out["y"] = y
    else:
        out["y8"], out["scale"] = y8, scale
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "linear": _own_linear, "sample": _own_sample,
                "norm": _own_norm}[op](state)
    return {"route": _plain_route, "linear": _plain_linear, "sample": _plain_sample,
            "norm": _plain_norm}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # logits in; indices, weights, both permutations and the maps out
        maps = sum(8 * (T * k // rows + min(E, T * k)) for rows in (32, 128))
        return {"bytes": 4 * T * E + 16 * T * k + maps + 8 * E, "flops": 4 * T * E}
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        size = 4 if case["out"] == "float32" else 2
        return {"bytes": N * K // 2 + 4 * N * (K // GROUP) + 2 * T * K + size * T * N,
                "flops": 2 * T * N * K}
    if op == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": 4 * B * V + 28 * B, "flops": 4 * B * V}
    T, d = case["T"], case["d"]
    res = {"none": 0, "bfloat16": 4, "float32": 8}[case["residual"]]
    size = 2 if case["out"] == "bfloat16" else 1 + 4 / GROUP
    return {"bytes": T * d * (2 + res + size) + 2 * d, "flops": 6 * T * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(s):
    c, E, k = s["case"], s["case"]["E"], s["case"]["k"]
    l = s["logits"].cpu().numpy().astype(np.float64)
    T = l.shape[0]
    if c["score"] == "softmax":
        z = np.exp(l - l.max(1)[:, None])
        score = z / z.sum(1)[:, None]
    else:
        score = np.where(l >= 0, 1.0, np.exp(np.minimum(l, 0.0))) / (1.0 + np.exp(-np.abs(l)))
    sel = score.copy()
    if s["balance"] is not None:
        sel += s["balance"].cpu().numpy().astype(np.float64)[None]
    if c["groups"] > 1:
        G = c["groups"]
        best = np.sort(sel.reshape(T, G, -1), 2)[:, :, ::-1][:, :, :c["group_top"]].sum(2)
        rank = np.argsort(np.argsort(-best, 1, kind="stable"), 1)
        sel = np.where(np.repeat(rank < c["keep"], E // G, 1), sel, -np.inf)
    idx = np.argsort(-sel, 1, kind="stable")[:, :k]
    w = np.take_along_axis(score, idx, 1)
    if c["renorm"]:
        w = w / w.sum(1)[:, None]
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    perm = np.argsort(flat, kind="stable")
    inv = np.argsort(perm, kind="stable")
    out = {"idx": idx, "w": w * c["scale"], "counts": counts, "offsets": offsets, "perm": perm,
           "inv_perm": inv}
    for rows, m, n in ((32, "block_map", "n_blocks"), (128, "tile_map", "n_tiles")):
        tiles = np.zeros((T * k // rows + min(E, T * k), 2), np.int64)
        per = -(-counts // rows)
        e = np.repeat(np.arange(E), per)
        j = np.arange(e.size) - np.repeat(np.cumsum(per) - per, per)
        tiles[:e.size, 0], tiles[:e.size, 1] = e, offsets[e] + rows * j
        out[m], out[n] = tiles, np.array([e.size])
    return {name: v if name == "w" else v.astype(np.int32) for name, v in out.items()}


def _exact_linear(s):
    q, x = s["q"], s["x"].double()
    N, words = q.shape
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 26) // (8 * words))
    for n in range(0, N, step):
        part = q[n:n + step].long() & 0xFFFFFFFF
        w = torch.empty((part.shape[0], words, 8), dtype=torch.float64, device=x.device)
        for i in range(8):
            w[:, :, i] = ((part >> (4 * i)) % 16).double()
        w = w.view(part.shape[0], -1, GROUP)
        w = w * s["scale"][n:n + step].double()[:, :, None]
        w = w + s["bias"][n:n + step].double()[:, :, None]
        # codes and scales of this range make sums that fit fp32, so this rounds once
        w = w.float().to(torch.bfloat16).double().view(part.shape[0], -1)
        out[:, n:n + step] = torch.mm(x, w.t().contiguous())
    return out


def _exact_sample(s):
    host = {n: s[n].cpu().numpy() for n in ("logits", "u", "temperature", "top_k", "top_p",
                                            "min_p")}
    tokens, probs = [], []
    for b, row in enumerate(host["logits"].astype(np.float64)):
        V, temp = row.size, float(host["temperature"][b])
        order = np.argsort(-row, kind="stable")
        if temp <= 0:
            tokens.append(order[0])
            probs.append(1.0)
            continue
        weight = np.exp((row[order] - row[order[0]]) / temp)
        n = int(host["top_k"][b])
        n = V if n <= 0 or n > V else n
        if host["top_p"][b] < 1:
            mass = np.cumsum(weight[:n])
            n = 1 + int(np.searchsorted(mass, float(host["top_p"][b]) * mass[-1], side="left"))
        n = max(1, min(n, int((weight >= float(host["min_p"][b])).sum())))
        kept = np.sort(order[:n])
        cum = np.cumsum(np.exp((row[kept] - row[order[0]]) / temp))
        at = np.searchsorted(cum, float(host["u"][b]) * cum[-1], side="right")
        tokens.append(kept[min(int(at), n - 1)])
        probs.append(float(np.diff(cum, prepend=0.0)[min(int(at), n - 1)] / cum[-1]))
    return {"token": np.array(tokens, np.int32), "prob": np.array(probs)}


def _exact_norm(s):
    c, out = s["case"], {}
    v = s["x"].double()
    if s["residual"] is not None:
        v = v + s["residual"].double()
        out["residual"] = v
        # the norm is of the residual as it is stored
        v = v.float().to(s["residual"].dtype).double()
    w = s["weight"].double() + float(c["plus_one"])
    y = w * v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + 1e-6)
    if c["out"] == "bfloat16":
        out["y"] = y
    else:
        scale = y.abs().reshape(y.shape[0], -1, GROUP).max(2).values / E4M3_MAX
        out["y8"] = y / torch.repeat_interleave(scale, GROUP, 1).clamp(min=1e-300)
        out["scale"] = scale
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"route": _exact_route, "linear": _exact_linear, "sample": _exact_sample,
            "norm": _exact_norm}[case["op"]](s)
