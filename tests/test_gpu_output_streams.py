"""Calls on a stream of their own that make their outputs: neither a block that the current stream has yet to read nor one
that it has been given in the meantime is written."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
import synth
from helpers import make_layer

pytestmark = pytest.mark.gpu

T, H = 1536, 2048                     # outputs of 12 MB (bf16: 6 MB), each a block of its own
SLEEP = 100_000_000                   # clocks, about 50 ms


def _ops():
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, 64, generator=gen, device="cuda").bfloat16()
    w = torch.randn(1, H, 64, generator=gen, device="cuda").bfloat16()
    grouped = moe.GroupedExperts(w)
    q = torch.randint(0, 256, (1, H, 32), generator=gen, device="cuda", dtype=torch.uint8)
    four = moe.W4Experts(q, torch.rand(1, H, 2, generator=gen, device="cuda").half(), group=32)
    y = torch.randn(T, H, generator=gen, device="cuda")
    norm = moe.NormResidual(H, gamma_pre=torch.rand(H, generator=gen, device="cuda"))
    return {"grouped": (lambda s: [grouped(x, stream=s)]), "w4": (lambda s: [four(x, stream=s)]),
            "norm": (lambda s: list(norm(y, y, stream=s)))}


@pytest.fixture(scope="module")
def ops():
    made = _ops()
    tl = make_layer(synth.DECODE, 3, T)
    layer, x = tl.moe_layer(), tl.x.cuda()
    made["layer"] = lambda s: [layer(x, stream=s)]
    return made


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["grouped", "w4", "norm", "layer"])
def test_made_outputs_do_not_meet_the_current_stream_s_blocks(ops, name, handle):
    run = ops[name]
    want = [t.clone() for t in run(None)]
    shapes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    run(s)                                           # (the stream's own memory and the layer's workspace are there)
    torch.cuda.synchronize()
    # blocks that the current stream frees before it has read them
    old = [torch.full(shape, 3.0, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in old]
    del old
    got = run(s)
    torch.cuda.synchronize()
    assert all(bool((t == 3.0).all()) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # outputs that are dropped while the stream has yet to write them
    del got
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = run(s)
    del got
    new = [torch.full(shape, 5.0, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    assert all(bool((t == 5.0).all()) for t in new)


def test_a_dropped_layer_s_workspace_is_not_given_away_while_a_stream_writes_it():
    tl = make_layer(synth.DECODE, 3, T)
    x = tl.x.cuda()
    layer = tl.moe_layer()
    nbytes = layer.ensure_workspace(T).numel()       # (memory of the current stream)
    side = torch.cuda.Stream()
    out = layer(x, stream=side)
    torch.cuda.synchronize()
    want = out.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    out = layer(x, stream=side)
    layer.ws, layer.ws_T = None, -1                  # (as a larger workspace or the end of the layer does)
    new = torch.full((nbytes,), 5, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((new == 5).all()) and torch.equal(out, want)
