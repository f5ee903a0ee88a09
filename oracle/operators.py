"""The operators around the layer in 64 bits, one row at a time, from their
definitions (numpy only; test infrastructure like the rest of this package)."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def sort_assignments(idx, E: int) -> dict:
    """counts, offsets, perm, inv_perm of selections idx [T, k] in stable expert order."""
    flat = np.asarray(idx).reshape(-1)
    counts = np.bincount(flat, minlength=E)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(flat.size)
    return {"counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]), "perm": perm,
            "inv_perm": inv}


def tiles(counts, rows: int) -> np.ndarray:
    """(expert, first sorted row) of every tile of `rows` rows, experts ascending."""
    out, row = [], 0
    for e, c in enumerate(counts):
        out += [(e, row + j) for j in range(0, int(c), rows)]
        row += int(c)
    return np.array(out, np.int64).reshape(-1, 2)


def route_scored(logits, k: int, score="softmax", balance=None, n_groups=1, top_groups=1,
                 group_top=1, renorm=True, scale=1.0):
    """(idx [T, k], w [T, k]) of the scored routing."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    bal = np.zeros(E) if balance is None else np.asarray(balance, np.float64)
    idx, w = np.empty((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = l > -np.inf  # (NaN compares false)
        s = np.zeros(E)
        if score == "sigmoid":
            e = np.exp(-np.minimum(np.abs(l[live]), 800.0)) * (np.abs(l[live]) <= 700.0)
            s[live] = np.where(l[live] >= 0, 1.0, e) / (1.0 + e)
        elif live.any():
            m = l[live].max()
            z = np.array([0.0 if not ok else 1.0 if v == m else np.exp(v - m) if m - v <= 700.0 else 0.0
                          for v, ok in zip(l, live)])
            s = z / z.sum()
        live &= np.isfinite(bal)
        v = np.where(live, s + np.where(np.isfinite(bal), bal, 0.0), -np.inf)
        part = np.ones(E, bool)
        if n_groups > 1:
            per = E // n_groups
            g = []
            for j in range(n_groups):
                best = np.sort(v[j * per:(j + 1) * per])[::-1][:group_top]
                best = best[best > -np.inf]
                g.append(best.sum() if best.size else -np.inf)
            keep = np.argsort(-np.array(g), kind="stable")[:top_groups]
            part[:] = False
            for j in keep:
                part[j * per:(j + 1) * per] = True
        cand = np.flatnonzero(part)
        pick = cand[np.argsort(-v[cand], kind="stable")][:k]
        idx[t] = pick
        wt = np.where(v[pick] > -np.inf, s[pick], 0.0)
        if renorm:
            wt = wt / wt.sum() if wt.sum() > 0 else np.zeros(k)
        w[t] = wt * scale
    return idx, w


def linear(q, scale, bias, x):
    """x [T, K] (float64) times the transposed matrix of bf16 weights bf16(q * scale + bias)."""
    from . import dequant
    w = (dequant(q, scale, bias).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return np.asarray(x, np.float64) @ w.T


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob) of one row, with weights in units of 2^-43 as exact integers, the
    token's own in prob unrounded; the parameters are fp32 values."""
    l = np.asarray(logits, np.float32).astype(np.float64)
    u, temperature, top_p, min_p = (float(np.float32(v)) for v in (u, temperature, top_p, min_p))
    V = l.size
    greedy = not temperature > 0
    t = 1.0 if greedy else float(temperature)
    k = 1 if greedy else V if top_k <= 0 or top_k > V else int(top_k)
    live = l > -np.inf
    if not live.any():
        return 0, 0.0
    big = float(np.finfo(np.float32).max)
    m = min(l[live].max(), big)
    w = np.zeros(V)
    with np.errstate(invalid="ignore", over="ignore"):
        x = (m - np.minimum(l[live], big)) / t
    w[live] = np.where(x < 30.4, np.exp(-x), 0.0)
    w = np.floor(w * 2.0 ** 43 + 0.5).astype(np.uint64)
    order = np.lexsort((np.arange(V), -np.where(live, l, -np.inf)))
    order = order[w[order] > 0][:k]
    if not greedy and top_p < 1:
        cum = np.cumsum(w[order])
        need = max(1, math.ceil(Fraction(max(float(top_p), 0.0)) * int(cum[-1])))
        order = order[:int(np.searchsorted(cum, np.uint64(int(need)), side="left")) + 1]
    if min_p > 0:
        order = order[w[order] >= np.ceil(min(float(min_p), 1.0) * 2.0 ** 43)]
    kept = np.sort(order)
    cum = np.cumsum(w[kept])
    total = int(cum[-1])
    draw = min(int(Fraction(max(float(u), 0.0)) * total), total - 1)
    at = int(np.searchsorted(cum, np.uint64(draw), side="right"))
    token = int(kept[at])
    return token, math.exp((min(l[token], big) - m) / t) * 2.0 ** 43 / total


BLOCK = 128  # columns (and weight rows) that share a scale of the 8-bit products


def expand(scale, rows: int, n: int, k: int) -> np.ndarray:
    """[n, k] in 64 bits: the scale of every element of a matrix with one per rows x 128."""
    s = np.asarray(scale, np.float64)
    return np.repeat(np.repeat(s, rows, 0)[:n], BLOCK, 1)[:, :k]


def product(w, w_scale, x, x_scale):
    """(y, the sum of the terms' magnitudes) of values w [N, K] and x [T, K] with their
    scales, in 64 bits."""
    wv = np.asarray(w, np.float64) * expand(w_scale, BLOCK, *w.shape)
    xv = np.asarray(x, np.float64) * expand(x_scale, 1, *x.shape)
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def group_scales(h) -> np.ndarray:
    """max |h| / 448 of every 128 columns."""
    n = h.shape[1]
    return np.stack([np.abs(h[:, j:j + BLOCK]).max(1) for j in range(0, n, BLOCK)], 1) / 448.0


def combine(rows, inv, w=None, base=None):
    """y [T, d] of expert rows [T k, d] with inv [T, k]; slots of weight 0 are left out."""
    T, k = inv.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for s in range(k):
            if w is None or w[t, s] != 0:
                y[t] += (1.0 if w is None else float(w[t, s])) * rows[inv[t, s]]
    return y if base is None else y + base


def combine_grad(dy, rows, inv, w):
    """(d_rows, d_w) of combine."""
    T, k = inv.shape
    d_rows, d_w = np.empty_like(rows), np.empty((T, k))
    for t in range(T):
        for s in range(k):
            d_rows[inv[t, s]] = float(w[t, s]) * dy[t]
            d_w[t, s] = (rows[inv[t, s]] * dy[t]).sum()
    return d_rows, d_w


def penalize(logits, tokens=(), n_prompt=0, repetition=1.0, frequency=0.0, presence=0.0,
             bias_ids=(), bias=(), allowed=None):
    """(out, the sum of the terms' magnitudes) of one row of logits; tokens: those that count."""
    y = np.asarray(logits, np.float32).astype(np.float64)
    V = y.size
    rep, freq, pres = (float(np.float32(v)) for v in (repetition, frequency, presence))
    rep = rep if rep > 0 else 1.0
    toks = [(i, int(v)) for i, v in enumerate(tokens) if 0 <= int(v) < V]
    for v in {v for _, v in toks}:
        y[v] = y[v] / rep if y[v] > 0 else y[v] * rep
    size = np.abs(y)
    count = {}
    for i, v in toks:
        if i >= n_prompt:
            count[v] = count.get(v, 0) + 1
    for v, n in count.items():
        y[v] -= freq * n + pres
        size[v] += abs(freq) * n + abs(pres)
    for v, b in zip(bias_ids, bias):
        if 0 <= int(v) < V:
            y[int(v)] += float(np.float32(b))
            size[int(v)] += abs(float(np.float32(b)))
    if allowed is not None:
        y[~np.asarray(allowed, bool)] = -np.inf
    return y, size
