"""Activations of the dense product's fp32 outputs over their range, at the accuracy that the header gives.

z is the bias alone (the weights are 0), which is exact.  In units of u = 2^-24, relative: the exponential's instruction 4
(2^-22), its argument's rest and product 1; reciprocal 2 (2^-23) and its sum 1; GELU's polynomial and its t 6; products 3: at
most 14, within 16 u = 2^-20.  The tanh form takes its exponent w = 2 sqrt(2 / pi) (z + 0.044715 z^3) rounded: with both
constants' roundings (0.58 and 0.48 u), three products and a sum w is off by at most 5.1 u relative, e^-|w| by
5.1 |w| u.  Above 0 that is damped by e^-|w| (5.1 w e^-w <= 1.9 u); below 0 it is the result's.
Results that are subnormal are rounded to their spacing of 2^-149 once more.
"""
from __future__ import annotations

import math

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FORM = 2 * math.sqrt(2 / math.pi)


def _silu(z):
    # (1 / (1 + e^-z) without an overflow)
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, z / (1 + e), z * e / (1 + e))


def _tanh_form(z):
    e = torch.exp(-(FORM * (z + 0.044715 * z ** 3)).abs())
    return torch.where(z >= 0, z / (1 + e), z * e / (1 + e))


ACTS = {"silu": _silu, "gelu": lambda z: 0.5 * z * torch.erfc(z * -math.sqrt(0.5)), "gelu_tanh": _tanh_form}


def _z(n):
    wide, near = torch.linspace(-120, 120, n // 2), torch.linspace(-8, 8, n // 4)
    small = torch.logspace(-30, 1, n - n // 2 - n // 4) * torch.tensor([1.0, -1.0]).repeat(n)[: n - n // 2 - n // 4]
    return torch.cat([wide, near, small]).float().cuda()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T, n, path", [(3, 8004, "split"), (2100, 2403, "pairs")])
def test_fp32_activations_over_their_range(act, T, n, path):
    bias = _z(n)
    op = moe.Linear(torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda"), bias, act=act, y_dtype=torch.float32)
    assert op.path(T) == path
    got = op(torch.ones(T, 8, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(got, got[:1].expand_as(got))        # (the same code whatever the row)
    z = bias.double()
    want = ACTS[act](z)
    rel = torch.full_like(z, 16 * U)
    if act == "gelu_tanh":
        rel = rel + torch.where(z < 0, 5.1 * U * (FORM * (z + 0.044715 * z ** 3)).abs(), torch.zeros_like(z))
    over = (got[0].double() - want).abs() - (rel * want.abs() + 2.0 ** -149)
    assert bool((over <= 0).all()), (over.max(), z[over.argmax()])
