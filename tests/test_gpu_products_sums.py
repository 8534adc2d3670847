"""Long sums of the grouped products with fp32 outputs: the error does not grow with the number of matrix instructions.

Tolerance, relative in norm, before any run.  An instruction that cuts its sum off loses half a unit on average, a unit is
at most 2^-23 of the partial sum, and partial sums of a run have 2/3 of its length's norm on average: a run of n
instructions is off by at most n * 2^-24 * 2 / 3 of its sum, and so is a sum of such runs.  n is at most 48 (gated: 24) in the
tensor kernel and 8 in the rows kernel.  Adding up to 19 runs with rounding, the join of 8 warps and the terms inside an instruction give at most
32 * 2^-24 / 4 more (errors of either sign: the root of their number).  The gated pair has the error of both sums, g's passing through silu, whose
relative slope g silu'(g) / silu(g) is at most 1.3 in norm for g of unit variance, and 8 roundings behind them.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [768, 776, 2048, 4099, 7168])
@pytest.mark.parametrize("T", [4, 40, 300])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("order", ["out_in", "in_out"])
@pytest.mark.parametrize("gather", [False, True])
def test_long_sums_keep_their_precision(K, T, up, order, gather):
    gen = torch.Generator(device="cuda").manual_seed(K + T)
    E, N = 3, 200
    pad = (-K) % 8
    cols = N + (-N) % 8
    make = lambda: torch.randn(E, N, K, generator=gen, device="cuda").bfloat16()
    w = [make() for _ in range(1 + up)]
    if order == "out_in":
        st = [torch.nn.functional.pad(v, (0, pad))[:, :, :K] for v in w]
    else:
        st = [torch.nn.functional.pad(v.transpose(1, 2).contiguous(), (0, cols - N))[:, :, :N] for v in w]
    k = 2 if gather else 1
    P = T * k
    sizes = [P - P // 3, 0, P // 3]
    off = torch.tensor([0, sizes[0], sizes[0], P], dtype=torch.int32, device="cuda")
    x = torch.nn.functional.pad((torch.randn(T, K, generator=gen, device="cuda") / K ** 0.5).bfloat16(), (0, pad))[:, :K]
    pairs = torch.randperm(P, generator=gen, device="cuda").int() if gather else None
    rows = (x[(pairs // k).long()] if gather else x).double()
    op = moe.GroupedExperts(st[0], st[1] if up else None, order=order)
    y = op(x, off, pairs, k=k)
    of = lambda v: torch.cat([rows[:sizes[0]] @ v[0].double().T, rows[sizes[0]:] @ v[2].double().T])
    g = of(w[0])
    exact = g / (1 + (-g).exp()) * of(w[1]) if up else g
    one = lambda n: n * 2.0 ** -24 * 2 / 3 + 8 * 2.0 ** -24
    n = 8 if op.path(T, k) == "rows" else 24 if up else 48
    bound = (1 + 1.3) * one(n) + 8 * 2.0 ** -24 if up else one(n)
    assert ((y.double() - exact).norm() / exact.norm()).item() <= bound
