"""Long sums of the grouped products with 16-bit outputs: the error stays that of the output's rounding at any n_in.

Tolerance, in norm, before any run.  A run has at most 8192 elements, 512 matrix instructions; each cuts off half a unit
on average, a unit is at most 2^-23 of the partial sum, and partial sums of a run have 2/3 of its length's norm on
average: 512 * 2^-24 * 2 / 3 of the run's sum, and so of a sum of runs.  Adding the runs and the terms inside an
instruction add at most 8 * 2^-24 (errors of either sign).  The gated pair has the error of both sums, g's passing
through silu, whose relative slope is at most 1.3 in norm for g of unit variance; exp, the division and the product add
8 * 2^-24 and, for g of at most 6 in magnitude, exp's 9 units of 2^-23.  What is stored is rounded: its error is that of
rounding the exact values, whose norm over the 8192 outputs another set of values of the same distribution meets to
within 5 % (the standard deviation of the sum of 8192 squared errors is 1 %, of its root half that).
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

HF, BF = torch.float16, torch.bfloat16


@pytest.mark.parametrize("K, up, order, dtype, y_dtype", [
    (8192, False, "out_in", HF, HF),             # one run
    (8200, True, "in_out", HF, HF),              # two, the second one shorter
    (8200, False, "out_in", BF, BF),
    (24584, True, "out_in", HF, HF),
    (1 << 18, False, "out_in", HF, HF),
    (1 << 18, True, "out_in", HF, HF),
    (1 << 18, False, "in_out", HF, HF),
    (1 << 20, True, "in_out", BF, BF),
    (1 << 20, False, "out_in", BF, BF),
])
@pytest.mark.parametrize("gather", [False, True])
def test_long_sums_end_in_one_rounding(K, up, order, dtype, y_dtype, gather):
    gen = torch.Generator(device="cuda").manual_seed(K % 1000 + up)
    E, N, T = 2, 96, 88                          # 88 rows of one expert, none of the other
    make = lambda: torch.empty(E, N, K, device="cuda", dtype=dtype).normal_(0, 1, generator=gen)
    w = [make() for _ in range(1 + up)]
    st = w if order == "out_in" else [v.transpose(1, 2).contiguous() for v in w]
    x = (torch.randn(T, K, generator=gen, device="cuda") / K ** 0.5).to(dtype)
    off = torch.tensor([0, 0, T], dtype=torch.int32, device="cuda")
    pairs = torch.randperm(T, generator=gen, device="cuda").int() if gather else None
    op = moe.GroupedExperts(st[0], st[1] if up else None, order=order, y_dtype=y_dtype)
    assert op.path(T) == "tensor"
    y = op(x, off, pairs)
    rows = (x[pairs.long()] if gather else x).double()
    of = lambda v: sum(rows[:, c:c + 65536] @ v[1, :, c:c + 65536].double().T for c in range(0, K, 65536))
    g = of(w[0])
    assert g.abs().max().item() <= 6
    exact = g / (1 + (-g).exp()) * of(w[1]) if up else g
    one = 512 * 2.0 ** -24 * 2 / 3 + 8 * 2.0 ** -24
    bound = (1 + 1.3) * one + 8 * 2.0 ** -24 + 9 * 2.0 ** -23 if up else one
    rounding = (exact.to(y_dtype).double() - exact).norm()
    assert ((y.double() - exact).norm() / exact.norm()).item() <= (1.05 * rounding / exact.norm()).item() + bound
    assert torch.equal(op(x, off, pairs), y)
