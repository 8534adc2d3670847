"""A launch that fails is reported by its own call and by no later one.

The failing launch goes to a stream whose capture has been invalidated (a synchronisation of the context in the middle of it),
which the runtime refuses on the host.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

pytestmark = pytest.mark.gpu


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(40, 64, device="cuda", generator=gen)
    xb = x.bfloat16()
    norm = moe.NormResidual(64, gamma_pre=torch.ones(64, device="cuda"))
    grouped = moe.GroupedExperts(torch.randn(1, 48, 64, device="cuda", generator=gen).bfloat16())
    q = torch.randint(0, 256, (1, 48, 32), dtype=torch.uint8, device="cuda", generator=gen)
    four = moe.W4Experts(q, torch.rand(1, 48, 2, device="cuda", generator=gen).half(), group=32)
    g, u, r = torch.ones(64, device="cuda"), torch.empty_like(xb), torch.empty_like(x)
    y, few = torch.empty(40, 48, device="cuda"), torch.empty(2, 48, device="cuda")
    return {"norm": lambda s: norm(x, x, x_out=r, u=u, stream=s), "rows": lambda s: grouped(xb[:2], out=few, stream=s),
            "tensor": lambda s: grouped(xb, out=y, stream=s), "w4": lambda s: four(xb, out=y, stream=s),
            "rmsnorm": lambda s: moe.moe_rmsnorm_bf16(x, g, 40, 64, 1e-6, u, s)}


@pytest.mark.parametrize("name", ["norm", "rows", "tensor", "w4", "rmsnorm"])
def test_a_failed_launch_is_reported_once(name):
    calls = _calls()
    for call in calls.values():
        call(None)
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 1) == 0                    # (non-blocking)
    try:
        assert cu.cuStreamBeginCapture_v2(stream, 0) == 0                     # (global: unsafe calls invalidate it)
        assert cu.cuCtxSynchronize() != 0
        with pytest.raises(N.MoeError) as ei:
            calls[name](stream.value)
        assert ei.value.status == N.MOE_ERR_CUDA
        assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    finally:
        cu.cuStreamDestroy_v2(stream)
    for call in calls.values():                                              # none of them fails for it
        call(None)
    torch.cuda.synchronize()
