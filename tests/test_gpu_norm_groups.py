"""add_norm with a scale per 128 columns against the formula in 64 bits.

Bars as for groups of 64: y is one fp32 value off by at most 2^-17 relative (the sum of
squares and six roundings); the scale likewise; codes half an e4m3 step, 2^-4 of the value or
2^-10 of the scale."""
import numpy as np
import pytest
import torch

import q4_routed_expert_amd as q4
from oracle import operators as plain
from routings import values

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -17


@pytest.mark.parametrize("T,d", [(1, 64), (1, 2048), (3, 192), (5, 448), (2, 576), (9, 1088),
                                 (4, 2112), (3, 4160), (2, 8192), (700, 1024)])
def test_groups_of_128(T, d):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16)
    if T > 1:
        x[1] = 0
    v = x.double().numpy()
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * w.double().numpy()
    y, y8, scale = q4.add_norm(x.cuda(), w.cuda(), e4m3=True, group=128)
    assert y is None and scale.shape == (T, -(-d // 128))
    s, got = plain.group_scales(want), scale.cpu().double().numpy()
    assert (np.abs(got - s) <= s * F32 + 2.0 ** -149).all()
    full = plain.expand(got, 1, T, d)
    bar = np.maximum(np.abs(want) * 2.0 ** -4, full * 2.0 ** -10) + 2 * F32 * np.abs(want)
    assert (np.abs(values(y8) * full - want) <= bar).all()
    # the codes and scales of groups of 64 stay what they were, the bf16 output is the same
    a = q4.add_norm(x.cuda(), w.cuda(), e4m3=True, y=torch.empty_like(x, device="cuda"))
    b = q4.add_norm(x.cuda(), w.cuda(), e4m3=True, group=128, y=torch.empty_like(x, device="cuda"))
    assert torch.equal(a[0], b[0]) and a[2].shape == (T, d // 64)
    pairs = torch.nn.functional.pad(a[2], (0, (d // 64) % 2)).view(T, -1, 2).amax(2)
    assert torch.equal(pairs, b[2])
