"""Routings and 8-bit inputs of the tests, made on the host without the library's kernels."""
import numpy as np
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain


def selections(rng, T, E, k, skew=0.5):
    """idx [T, k] (distinct in a row) and weights [T, k]; some experts come often, some never."""
    l = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    idx = np.argsort(-l, 1, kind="stable")[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32) + 0.1
    return idx, w / w.sum(1, keepdims=True)


def device_routing(idx, w, E, dev, room=0):
    """A DeviceRouting of the selections (for `room` more tokens than it holds)."""
    T, k = idx.shape
    o = plain.sort_assignments(idx, E)
    r = q4.DeviceRouting(T + room, E, k, dev)

    def put(t, a):
        a = torch.from_numpy(np.ascontiguousarray(a)).to(t.dtype)
        t.view(-1)[:a.numel()].copy_(a.view(-1))

    put(r.topk_idx, idx)
    put(r.topk_w, w)
    for name in ("counts", "offsets", "perm", "inv_perm"):
        put(getattr(r, name), o[name])
    for rows, m, n in ((32, r.block_map, r.n_blocks), (128, r.tile_map, r.n_tiles)):
        tiles = plain.tiles(o["counts"], rows)
        put(m, tiles)
        put(n, np.array([len(tiles)]))
    return r, o


def quantised_rows(rng, T, K, spread=1.0):
    """x [T, K] as e4m3 codes with a scale per 128 columns (tensors on the host)."""
    x = rng.standard_normal((T, K)) * np.exp(spread * rng.standard_normal((T, 1)))
    s = np.maximum(plain.group_scales(x), 1e-30).astype(np.float32)
    codes = torch.from_numpy(np.clip(x / plain.expand(s, 1, T, K), -448, 448)).to(torch.float32)
    return codes.to(torch.float8_e4m3fn), torch.from_numpy(s)


def values(codes):
    """e4m3 codes as a 64-bit array."""
    return codes.cpu().float().numpy().astype(np.float64)
