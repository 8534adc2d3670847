"""The norm over as many rows as T can name."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 8])
def test_norm_over_the_most_rows(T):
    """One element a row, so that a row's norm is its sign: exact in every step."""
    y = torch.ones(T, 1, dtype=torch.float16, device="cuda")
    y[::7] = -3.0
    op = moe.NormResidual(1, gamma_post=torch.full((1,), 2.0, device="cuda"), eps=0.0)
    out, u = op(None, y)
    assert u is None
    assert torch.equal(out, y.clamp_(-1, 1).mul_(2.0))
