"""Dense product, layer norm and balance loss on a stream of their own: what a call makes (workspaces too) is that stream's memory, and
a launch that fails is reported by its own call only."""
from __future__ import annotations

import ctypes

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

pytestmark = pytest.mark.gpu

T, H = 1536, 2048                     # outputs of 12 MB (bf16: 6 MB), each a block of its own
SLEEP = 100_000_000                   # clocks, about 50 ms


@pytest.fixture(scope="module")
def ops():
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, g, w, xs = rand(T, H), rand(H), rand(H, 64).bfloat16(), rand(T, 64).bfloat16()
    linear, norm, balance = moe.Linear(w, y_dtype=torch.float32), moe.LayerNorm(H, gamma=g, beta=g), moe.BalanceLoss(64, 4)
    logits = rand(T, 64)
    ids = torch.topk(logits, 4).indices.int()
    _, mean, rstd = norm(x)
    return {"linear": lambda s: [linear(xs, residual=x, stream=s)], "norm": lambda s: list(norm(x, stream=s)),
            "backward": lambda s: list(norm.backward(x, x, mean, rstd, add=x, stream=s)),
            "balance": lambda s: list(balance(logits, ids, dlogits=True, stream=s))}


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["linear", "norm", "backward", "balance"])
def test_made_outputs_do_not_meet_the_current_stream_s_blocks(ops, name, handle):
    run = ops[name]
    want = [t.clone() for t in run(None)]
    shapes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    run(s)
    torch.cuda.synchronize()
    # blocks that the current stream frees before it has read them
    old = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in old]
    del old
    got = run(s)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # outputs that are dropped while the stream has yet to write them
    del got
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = run(s)
    del got
    new = [torch.full(shape, 5, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in new)


@pytest.mark.parametrize("name", ["linear", "norm", "backward", "balance"])
def test_a_failed_launch_is_reported_once(name):
    """The launch goes to a stream whose capture has been invalidated, which the runtime refuses on the host."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(40, 64, device="cuda", generator=gen)
    xb, g = x.bfloat16(), torch.ones(64, device="cuda")
    linear, norm, balance = moe.Linear(xb[:16].contiguous()), moe.LayerNorm(64, gamma=g, beta=g), moe.BalanceLoss(64, 4)
    ids = torch.topk(x, 4).indices.int()
    y, z, d = torch.empty(40, 16, device="cuda", dtype=torch.bfloat16), torch.empty_like(xb), torch.empty_like(x)
    _, mean, rstd = norm(x)
    dg, db = torch.empty_like(g), torch.empty_like(g)
    ln, bl = N.moe_layer_norm_desc(64, N.MOE_F32, N.MOE_BF16, g.data_ptr(), g.data_ptr(), 1e-5), balance._desc[0]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    loss, counts = torch.empty(1, device="cuda"), torch.empty(64, dtype=torch.int32, device="cuda")
    calls = {"linear": lambda s: linear(xb, out=y, stream=s), "norm": lambda s: norm(x, out=z, mean=mean, rstd=rstd, stream=s),
             "backward": lambda s: N.moe_layer_norm_backward(ln, xb, 64, x, 64, mean, rstd, None, 0, 40, d, 64, dg, db, 0, ws, 1 << 20, s),
             "balance": lambda s: N.moe_balance_loss(bl, x, 64, ids, 40, None, 1, None, None, loss, counts, d, 64, None, ws, 1 << 20, s)}
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
