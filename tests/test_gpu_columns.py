"""Inputs and outputs that are columns of one buffer: the bits of separate ones, and nothing else written."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("four", [False, True])
def test_products_from_columns_to_columns(T, swapped, four):
    K, N_ = 64, 72
    if four:
        q = torch.randint(0, 256, (1, N_, K // 2), dtype=torch.uint8, device="cuda", generator=_gen(1))
        op = moe.W4Experts(q, torch.rand(1, N_, K // 32, device="cuda", generator=_gen(2)).half(), group=32, y_dtype=BF)
    else:
        op = moe.GroupedExperts(torch.randn(1, N_, K, device="cuda", generator=_gen(1)).to(BF), y_dtype=BF)
    values = torch.randn(T, K, device="cuda", generator=_gen(3)).to(BF)
    buf = torch.full((T, 8 + K + N_), 7.0, dtype=BF, device="cuda")
    x, y = (buf[:, 8 + N_:], buf[:, :N_]) if swapped else (buf[:, 8: 8 + K], buf[:, 8 + K:])
    x.copy_(values)
    want = op(values)
    op(x, out=y)
    assert torch.equal(y, want) and torch.equal(x, values)
    gap = buf[:, N_: N_ + 8] if swapped else buf[:, :8]
    assert bool((gap == 7.0).all())


@pytest.mark.parametrize("T, H", [(1, 64), (9, 100), (130, 2048), (300, 7168)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_over_columns_of_one_buffer(T, H, dtype):
    op = moe.NormResidual(H, gamma_post=torch.rand(H, device="cuda", generator=_gen(1)),
                          gamma_pre=torch.rand(H, device="cuda", generator=_gen(2)), res_scale=0.5, scale=1.25)
    x0, y0 = (torch.randn(T, H, device="cuda", generator=_gen(s)).to(dtype) for s in (3, 4))
    gate0 = torch.rand(T, H, device="cuda", generator=_gen(5)) if dtype is F32 else None
    want_x, want_u = op(x0, y0, gate=gate0, u=torch.empty(T, H, dtype=dtype, device="cuda"))
    buf = torch.full((T, 5 * H + 8), 7.0, dtype=dtype, device="cuda")
    x, y, x_out, u, gate = (buf[:, i * H: (i + 1) * H] for i in (1, 3, 0, 2, 4))
    x.copy_(x0)
    y.copy_(y0)
    if gate0 is not None:
        gate.copy_(gate0)
    op(x, y, gate=gate if gate0 is not None else None, x_out=x_out, u=u)
    assert torch.equal(x_out, want_x) and torch.equal(u, want_u) and torch.equal(x, x0) and torch.equal(y, y0)
    assert bool((buf[:, 5 * H:] == 7.0).all())
