"""Sums of the 4-bit products with fp16 rows and fp32 outputs, against the formula in 64 bits.

Tolerance, relative in norm, before any run.  A group's sum is two chains of at most 4 matrix instructions, each off by
half a unit on average, a unit being at most 2^-23 of the partial sum, which is 2/3 of the chain's on average:
4 * 2^-24 * 2 / 3 of sum q x.  The codes of a symmetric group are 8 + d with d of about 2.6 in norm, so that sum is
up to 3.3 times the wanted sum d x: 9 * 2^-24.  Taking off the zero point, scaling and adding the groups are
roundings of either sign: 8 * 2^-24.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T, K, N, group", [(1, 2048, 7168, 64), (14, 1408, 428, 128), (8, 2080, 200, 32), (1, 256, 130, 128),
                                            (16, 7168, 300, 64)])
@pytest.mark.parametrize("seed", [0, 1, 2, 3])
def test_w4_sums_keep_their_precision(T, K, N, group, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.empty(1, N, K // group, group, device="cuda").normal_(0.0, 0.02, generator=gen)
    s = (w.abs().amax(3, keepdim=True) / 7).half()
    c = (w / s.float() + 8.0).round().clamp(0, 15).to(torch.uint8).view(1, N, K)
    x = torch.empty(T, K, device="cuda").normal_(0.0, 1.0, generator=gen).half()
    y = moe.W4Experts(c[..., 0::2] | (c[..., 1::2] << 4), s[..., 0], group=group, x_dtype=torch.float16)(x)
    exact = x.double() @ ((c.double() - 8).view(N, -1, group) * s[0].double()).view(N, K).T
    assert ((y.double() - exact).norm() / exact.norm()).item() <= 17 * 2.0 ** -24
