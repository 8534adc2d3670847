"""A wait of the 4-bit products that runs out where a CTA has many more steps than the ring has stages: the call ends within
the limit, says so, and the next call gives the bits of the one before.

Time, before any run: a wait tests its barrier 64 times, up to 0.1 ms each, before it looks at the clock, and then gives up
after the limit; the copies in flight are waited for within the limit and are long done.  What is left is the call itself
and its launch: less than a limit of 20 ms.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N
from test_gpu_products import _quantize

pytestmark = pytest.mark.gpu

LIMIT_NS = 20_000_000


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("up, zeros, aligned", [(False, True, True), (True, True, True), (True, False, True), (False, True, False)])
def test_w4_wait_that_runs_out_far_from_the_end(group, up, zeros, aligned):
    E, N_, K, T = 4, 10000, 1792, 6              # 316 units or more of 7 steps: 2 to 5 units a CTA
    gen = torch.Generator(device="cuda").manual_seed(group)

    def make():
        q, s, z = _quantize(torch.randn(E, N_, K, generator=gen, device="cuda") * 0.05, group, zeros)
        if not aligned:                          # (scales copied one by one)
            s = torch.empty(s.numel() + 1, dtype=s.dtype, device="cuda")[1:].view(s.shape).copy_(s)
        return q, s, z

    a, b = make(), (make() if up else None)
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, 1, 2, 4, 6], dtype=torch.int32, device="cuda")
    op = moe.W4Experts(*a, up=b, group=group)
    ref = op(x, off).clone()
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(ref)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    try:
        N.moe_debug_set_waits(LIMIT_NS, 1)
        t[0].record()
        op(x, off, out=out, status=status)
        t[1].record()
        torch.cuda.synchronize()
    finally:
        N.moe_debug_set_waits(0, 0)
    assert status.item() == N.MOE_ERR_TIMEOUT
    assert t[0].elapsed_time(t[1]) <= 64 * 0.1 + 2 * LIMIT_NS * 1e-6
    assert torch.equal(op(x, off), ref)
