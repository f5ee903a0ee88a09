"""Gradients of slots of weight 0, which combine leaves out whatever their rows hold (rows that
nothing has written, say): d_w stays finite, so that a router's backward pass can multiply it by 0."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from routings import device_routing, selections

pytestmark = pytest.mark.gpu


# rows of one lane group and of a work group, one and several pieces a thread
@pytest.mark.parametrize("T,E,k,d", [(9, 8, 4, 64), (9, 8, 4, 128), (7, 8, 3, 192), (5, 8, 2, 448),
                                     (6, 8, 4, 576), (5, 16, 8, 4160)])
def test_d_w_of_left_out_rows_is_finite(T, E, k, d):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(T + d)
    idx, w = selections(rng, T, E, k)
    r, o = device_routing(idx, w, E, dev)
    inv = o["inv_perm"].reshape(T, k)
    rows = torch.from_numpy(rng.standard_normal((T * k, d)).astype(np.float32)).to(torch.bfloat16)
    dy = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16)
    plain_rows, plain_w = (t.cpu() for t in q4.combine_grad(dy.to(dev), rows.to(dev), r))
    left_out = {(0, 0): float("nan"), (1, 1): float("inf"), (2, 0): 3e38, (3, 1): None}
    for (t, s), v in left_out.items():
        w[t, s] = 0.0
        if v is not None:
            rows[int(inv[t, s]), 1::7] = v   # (1, 1), (2, 0): sums of infinities of both signs
    rows[int(inv[4, 0]), 5] = float("nan")   # a slot that counts
    r.topk_w.copy_(torch.from_numpy(w))
    d_rows, d_w = (t.cpu() for t in q4.combine_grad(dy.to(dev), rows.to(dev), r))
    for (t, s), v in left_out.items():
        assert (d_rows[int(inv[t, s])] == 0).all()
        if v is None:                        # a finite row: the formula's, as for any weight
            assert d_w[t, s] == plain_w[t, s] != 0
        elif v != 3e38:
            assert d_w[t, s] == 0, (t, s, d_w[t, s])
        assert d_w[t, s].isfinite(), (t, s, d_w[t, s])
    assert d_w[4, 0].isnan()
    rest = [(t, s) for t in range(T) for s in range(k) if (t, s) not in left_out and (t, s) != (4, 0)]
    for t, s in rest:
        assert d_w[t, s] == plain_w[t, s] and torch.equal(d_rows[int(inv[t, s])], plain_rows[int(inv[t, s])])
