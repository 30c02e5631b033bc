"""Rotary positions at the most heads that the documentation allows."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import L, _rope_tol  # noqa: F401  (the library's fixture)

pytestmark = pytest.mark.gpu


def test_rope_most_heads(L, gpu):
    """2^20 heads, the documented most, of more columns than a row of threads takes at once."""
    n, h, d, first, rot = 1, 1 << 20, 259, 1, 2
    x = torch.randn((n, h, d), device=gpu).to(torch.bfloat16)
    pos, freqs = torch.tensor([12345], dtype=torch.int32, device=gpu), torch.tensor([1.0], dtype=torch.float64, device=gpu)
    got = L.rope_rotate(x, pos, freqs, first=first)
    some = [0, 1, 65535, 65536, (1 << 20) - 17, (1 << 20) - 1]
    assert torch.equal(got[..., :1], x[..., :1]) and torch.equal(got[..., 3:], x[..., 3:])
    x64 = x[:, some].double().cpu().numpy()
    ref = paged.rope_rotate(x64, [12345], [1.0], first)
    tol = _rope_tol(x64, ref, [12345], np.array([1.0]), first, rot, False, 1.0, True)
    assert (np.abs(got[:, some].double().cpu().numpy() - ref) <= tol).all()
    a, b = x[..., 1].double(), x[..., 2].double()
    turned = torch.stack([a * math.cos(12345) - b * math.sin(12345), a * math.sin(12345) + b * math.cos(12345)], -1)
    # a bf16 rounding, and products and an angle in fp32 (below 2^-18 of |a| + |b| together)
    tol = 2.0 ** -8 * turned.abs() + 2.0 ** -18 * (a.abs() + b.abs())[..., None]
    assert ((got[..., 1:3].double() - turned).abs() <= tol).all()
