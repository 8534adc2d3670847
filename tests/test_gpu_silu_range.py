"""The gated products over the whole range of g: silu(g) u where e^-g overflows, for g beyond every threshold, in each type
and kernel.

Tolerance, before any run.  Here g and u are single products, exact in fp32.  fp32 outputs, in units of 2^-24 of the result:
exp 4 (2 units in the last place), its product with g, 1 + z and the division 1 each, the product with u 1: 8.
16-bit outputs: half a step, and of the tensor kernel's quick exponential and division 2 (2 + 1.173 |g|) + 4 + 3 such units.  silu(g) is an fp32
number: e^-|g| and silu(g) are each off by up to 2^-149, so |u| (1 + |g|) 2^-149 more.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
G = [0.0, -0.0, 2.0 ** -20, -1.0, 1.0, -10.0, 10.0, -20.0, -40.0, -80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -92.0, -95.0, -100.0,
     -103.0, -104.0, -120.0, -1000.0, 40.0, 88.0, 89.0, 100.0, 1000.0]


@pytest.mark.parametrize("y_dtype", [F32, BF, HF])
@pytest.mark.parametrize("kernel, T", [("rows", 2), ("tensor", 40), ("w4", 2), ("w4", 12)])
@pytest.mark.parametrize("u", [1.0, -(2.0 ** 15), 2.0 ** 100])
def test_gated_products_over_the_range_of_g(kernel, T, y_dtype, u):
    if u == 2.0 ** 100 and y_dtype is HF:
        u = 2.0 ** 14
    N_, K = 32, 32
    g = torch.zeros(N_, dtype=F32)
    g[: len(G)] = torch.tensor(G)
    w = torch.zeros(1, N_, K, dtype=BF, device="cuda")
    w[0, :, 0] = g.to(BF)
    w_up = torch.zeros_like(w)
    w_up[0, :, 1] = u
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    x[:, :2] = 1.0
    if kernel == "w4":                           # a weight of 1 for g in column 0 and for u in column 1; g comes from the scale
        q = torch.full((1, N_, K // 2), 0x88, dtype=torch.uint8, device="cuda")
        qg, qu = q.clone(), q.clone()
        qg[:, :, 0], qu[:, :, 0] = 0x89, 0x98
        op = moe.W4Experts(qg, w[:, :, :1].contiguous(), up=(qu, w_up[:, :, 1:2].contiguous()), group=32, y_dtype=y_dtype)
    else:
        op = moe.GroupedExperts(w, w_up, y_dtype=y_dtype)
        assert op.path(T) == kernel
    y = op(x).double()
    gd = w[0, :, 0].double()
    want = torch.where(gd == 0, 0.0, gd * torch.where(gd < 0, gd, -gd).exp() ** (gd < 0) / (1 + (-gd.abs()).exp())) * u
    units = 8 + (2 * (2 + 1.173 * gd.abs()) + 7 if y_dtype is not F32 else 0)
    tol = units * 2.0 ** -24 * want.abs() + abs(u) * (1 + gd.abs()) * 2.0 ** -149
    if y_dtype is not F32:
        tol = tol + torch.finfo(y_dtype).eps / 2 * (want.abs() + tol)
    tol = tol + torch.finfo(y_dtype).smallest_normal * torch.finfo(y_dtype).eps
    top = torch.finfo(y_dtype).max
    want = torch.where(want.abs() > top, want.sign() * float("inf"), want)
    off = torch.where(torch.isinf(want), torch.where(y == want, -1.0, 1.0), (y - want).abs() - tol)
    assert bool((off <= 0).all()), [(gd[i].item(), y[r, i].item(), want[i].item()) for r, i in (off > 0).nonzero().tolist()[:8]]


@pytest.mark.parametrize("T", [2, 40])
def test_gated_products_of_what_is_not_finite(T):
    """g infinite or NaN: infinity times u, 0 times infinity is NaN as in the formula."""
    w = torch.zeros(1, 16, 8, dtype=BF, device="cuda")
    w[0, :3, 0] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    w_up = torch.zeros_like(w)
    w_up[0, :, 0] = 2.0
    x = torch.zeros(T, 8, dtype=BF, device="cuda")
    x[:, 0] = 1.0
    y = moe.GroupedExperts(w, w_up)(x)
    assert bool((y[:, 0] == float("inf")).all()) and bool(torch.isnan(y[:, 1:3]).all()) and bool((y[:, 3:] == 0).all())
