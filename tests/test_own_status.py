"""The status word of the products' wrappers: what a call without one raises can be asked for."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N
from test_products_devices import _args, ops  # noqa: F401


@pytest.mark.parametrize("which", [0, 1])
def test_calls_pass_their_own_word_unless_one_is_given(ops, which):  # noqa: F811
    op, calls = ops[which], ops[3]
    given = _args()
    op(**dict(given, status=None))
    op(**given)
    own, theirs = calls[0][9], calls[1][9]
    assert own is op._status and own.dtype is torch.int32 and own.numel() == 1 and theirs is given["status"]
    assert op.device_status() == N.MOE_OK
    own[0] = N.MOE_ERR_TIMEOUT
    assert op.device_status(clear=True) == N.MOE_ERR_TIMEOUT and op.device_status() == N.MOE_OK
    assert ops[1 - which]._status.data_ptr() != own.data_ptr()


def test_words_are_not_given_twice():
    words = [moe.layer._status_word(torch.device("cpu")) for _ in range(2500)]
    assert len({w.data_ptr() for w in words}) == 2500 and all(int(w) == N.MOE_OK for w in words)


def _made(four):
    gen = torch.Generator(device="cuda").manual_seed(3)
    if four:
        q = torch.randint(0, 256, (3, 40, 32), dtype=torch.uint8, device="cuda", generator=gen)
        return moe.W4Experts(q, torch.rand(3, 40, 2, device="cuda", generator=gen).half(), group=32)
    return moe.GroupedExperts(torch.randn(3, 40, 64, device="cuda", generator=gen).bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T", [4, 300])
def test_bad_routing_and_waits_that_ran_out_can_be_asked_for(T, four):
    op, other = _made(four), _made(four)
    x = torch.randn(T, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    good = torch.tensor([0, 1, T, T], dtype=torch.int32, device="cuda")
    ref = op(x, good).clone()
    assert op.device_status() == N.MOE_OK
    op(x, torch.tensor([0, 1, T, T + 1], dtype=torch.int32, device="cuda"))
    assert op.device_status() == N.MOE_ERR_DEVICE_CHECK and other.device_status() == N.MOE_OK
    op(x, good)
    assert op.device_status(clear=True) == N.MOE_ERR_DEVICE_CHECK and op.device_status() == N.MOE_OK
    if four or T == 300:                         # (the streaming kernel waits for nothing)
        try:
            N.moe_debug_set_waits(2_000_000, 1)
            op(x, good)
            torch.cuda.synchronize()
        finally:
            N.moe_debug_set_waits(0, 0)
        assert op.device_status(clear=True) == N.MOE_ERR_TIMEOUT
    assert torch.equal(op(x, good), ref) and op.device_status() == N.MOE_OK


@pytest.mark.gpu
def test_a_captured_call_raises_the_word_after_its_object_is_gone():
    op = _made(False)
    x = torch.randn(4, 64, device="cuda").bfloat16()
    off = torch.tensor([0, 1, 4, 4], dtype=torch.int32, device="cuda")
    y = torch.empty(4, 40, device="cuda")
    op(x, off, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(x, off, out=y)
    word, keep = op._status, op._keep
    del op
    torch.cuda.empty_cache()
    off[3] = 9
    graph.replay()
    torch.cuda.synchronize()
    assert word.item() == N.MOE_ERR_DEVICE_CHECK and keep is not None
