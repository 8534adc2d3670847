"""Refusals of the grouped, 4-bit and norm calls: bad arguments are named on the host, before any launch (no GPU)."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

FAKE = 0x100000
FAR = 0x4000000000          # another address, far from FAKE: nothing here is ever dereferenced


def _refused(status, word, fn, *args):
    with pytest.raises(N.MoeError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)
    assert word in str(ei.value), str(ei.value)


def _dense(**kw):
    d = dict(type=N.MOE_BF16, y_type=N.MOE_F32, order=N.MOE_W_OUT_IN, n_experts=4, n_out=48, n_in=64, w=FAKE, w_up=None,
             row_stride=64, expert_stride=48 * 64)
    d.update(kw)
    return N.moe_grouped_desc(*d.values())


@pytest.mark.parametrize("kw, status, word", [
    (dict(type=N.MOE_F32), N.MOE_ERR_UNSUPPORTED, "type"),
    (dict(type=N.MOE_Q4_K), N.MOE_ERR_UNSUPPORTED, "type"),
    (dict(y_type=N.MOE_Q8_0), N.MOE_ERR_UNSUPPORTED, "y_type"),
    (dict(order=2), N.MOE_ERR_INVALID_ARG, "order"),
    (dict(n_experts=0), N.MOE_ERR_INVALID_ARG, "n_experts"),
    (dict(n_experts=1025), N.MOE_ERR_INVALID_ARG, "n_experts"),
    (dict(n_out=0), N.MOE_ERR_INVALID_ARG, "n_out"),
    (dict(n_in=(1 << 20) + 1, row_stride=(1 << 20) + 8), N.MOE_ERR_INVALID_ARG, "n_in"),
    (dict(w=None), N.MOE_ERR_INVALID_ARG, "NULL"),
    (dict(w=FAKE + 8), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(w_up=FAKE + 2), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(row_stride=56), N.MOE_ERR_INVALID_ARG, "row_stride"),
    (dict(row_stride=68), N.MOE_ERR_INVALID_ARG, "row_stride"),
    (dict(expert_stride=47 * 64), N.MOE_ERR_INVALID_ARG, "expert_stride"),
    (dict(expert_stride=48 * 64 + 4), N.MOE_ERR_INVALID_ARG, "expert_stride"),
    (dict(order=N.MOE_W_IN_OUT, row_stride=40), N.MOE_ERR_INVALID_ARG, "row_stride"),
])
def test_grouped_plan_refusals(kw, status, word):
    _refused(status, word, moe.moe_grouped_plan_create, _dense(**kw))


_CALL = [
    (dict(T=-1), N.MOE_ERR_INVALID_ARG, "T = -1"),
    (dict(k=0), N.MOE_ERR_INVALID_ARG, "k = 0"),
    (dict(k=33), N.MOE_ERR_INVALID_ARG, "k = 33"),
    (dict(T=1 << 28, k=8), N.MOE_ERR_INVALID_ARG, "too large"),
    (dict(offsets=None), N.MOE_ERR_INVALID_ARG, "offsets"),
    (dict(x=None), N.MOE_ERR_INVALID_ARG, "NULL"),
    (dict(y=None), N.MOE_ERR_INVALID_ARG, "NULL"),
    (dict(x=FAKE + 8), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(y=FAR + 2), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(offsets=FAKE + 2), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(status=FAKE + 1), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(x_stride=56), N.MOE_ERR_INVALID_ARG, "x_stride"),
    (dict(x_stride=68), N.MOE_ERR_INVALID_ARG, "x_stride"),
    (dict(y_stride=47), N.MOE_ERR_INVALID_ARG, "y_stride"),
    (dict(y=FAKE + 256), N.MOE_ERR_INVALID_ARG, "overlaps"),
]


def _call(**kw):
    d = dict(x=FAKE, x_stride=64, T=3, k=2, sorted_pairs=None, offsets=FAKE, y=FAR, y_stride=48, status=None, stream=0)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw, status, word", _CALL)
def test_grouped_call_refusals(kw, status, word):
    plan = moe.moe_grouped_plan_create(_dense())
    try:
        _refused(status, word, moe.moe_grouped_matmul, plan, *_call(**kw))
        moe.moe_grouped_matmul(plan, *_call(T=0, x=None, y=None))          # no tokens: nothing launched
    finally:
        moe.moe_grouped_plan_destroy(plan)
    _refused(N.MOE_ERR_INVALID_ARG, "plan", moe.moe_grouped_matmul, None, *_call())


def _four(**kw):
    d = dict(x_type=N.MOE_BF16, y_type=N.MOE_F32, scale_type=N.MOE_F16, group=32, n_experts=4, n_out=48, n_in=64, q=FAKE,
             scales=FAKE, zeros=None, q_up=None, scales_up=None, zeros_up=None)
    d.update(kw)
    return N.moe_w4_desc(*d.values())


@pytest.mark.parametrize("kw, status, word", [
    (dict(x_type=N.MOE_F32), N.MOE_ERR_UNSUPPORTED, "x_type"),
    (dict(y_type=N.MOE_Q4_K), N.MOE_ERR_UNSUPPORTED, "y_type"),
    (dict(scale_type=N.MOE_F32), N.MOE_ERR_UNSUPPORTED, "scale_type"),
    (dict(group=16), N.MOE_ERR_UNSUPPORTED, "group"),
    (dict(group=128), N.MOE_ERR_INVALID_ARG, "multiple"),
    (dict(n_out=0), N.MOE_ERR_INVALID_ARG, "n_out"),
    (dict(n_experts=2000), N.MOE_ERR_INVALID_ARG, "n_experts"),
    (dict(q=None), N.MOE_ERR_INVALID_ARG, "NULL"),
    (dict(scales=None), N.MOE_ERR_INVALID_ARG, "NULL"),
    (dict(q=FAKE + 8), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(scales=FAKE + 1), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(q_up=FAKE), N.MOE_ERR_INVALID_ARG, "scales_up"),
    (dict(q_up=FAKE, scales_up=FAKE, zeros=FAKE), N.MOE_ERR_INVALID_ARG, "zeros_up"),
    (dict(zeros=FAKE, zeros_up=FAKE), N.MOE_ERR_INVALID_ARG, "zeros_up"),
])
def test_w4_plan_refusals(kw, status, word):
    _refused(status, word, moe.moe_w4_plan_create, _four(**kw))


@pytest.mark.parametrize("kw, status, word", _CALL)
def test_w4_call_refusals(kw, status, word):
    plan = moe.moe_w4_plan_create(_four())
    try:
        _refused(status, word, moe.moe_w4_matmul, plan, *_call(**kw))
        moe.moe_w4_matmul(plan, *_call(T=0, x=None, y=None))
    finally:
        moe.moe_w4_plan_destroy(plan)


def _norm(**kw):
    d = dict(H=64, x_type=N.MOE_F32, y_type=N.MOE_F32, u_type=N.MOE_BF16, gamma_post=FAKE, gamma_pre=FAKE, eps=1e-6,
             res_scale=1.0, scale=1.0)
    d.update({n: v for n, v in kw.items() if n in d})
    c = dict(x=FAKE, x_stride=64, y=FAR, y_stride=64, gate=None, gate_row=0, gate_col=0, T=4, x_out=2 * FAR, x_out_stride=64,
             u=3 * FAR, u_stride=64, stream=0)
    c.update({n: v for n, v in kw.items() if n in c})
    return [N.moe_norm_desc(*d.values())] + list(c.values())


@pytest.mark.parametrize("kw, status, word", [
    (dict(H=0), N.MOE_ERR_INVALID_ARG, "H = 0"),
    (dict(H=32769, x_stride=40000, y_stride=40000, x_out_stride=40000, u_stride=40000), N.MOE_ERR_INVALID_ARG, "H = 32769"),
    (dict(x_type=N.MOE_Q8_0), N.MOE_ERR_UNSUPPORTED, "types"),
    (dict(u_type=N.MOE_Q4_K), N.MOE_ERR_UNSUPPORTED, "types"),
    (dict(eps=-1e-6), N.MOE_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), N.MOE_ERR_INVALID_ARG, "eps"),
    (dict(T=-2), N.MOE_ERR_INVALID_ARG, "T = -2"),
    (dict(y=None), N.MOE_ERR_INVALID_ARG, "y is NULL"),
    (dict(gamma_pre=None), N.MOE_ERR_INVALID_ARG, "gamma_pre"),
    (dict(u=None, x_out=None), N.MOE_ERR_INVALID_ARG, "neither"),
    (dict(x_stride=63), N.MOE_ERR_INVALID_ARG, "stride"),
    (dict(y_stride=-64), N.MOE_ERR_INVALID_ARG, "stride"),
    (dict(gate=FAKE, gate_col=-1), N.MOE_ERR_INVALID_ARG, "gate"),
    (dict(x=FAKE + 2), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(gamma_post=FAKE + 2), N.MOE_ERR_INVALID_ARG, "aligned"),
    (dict(x_out=FAR + 64), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(u=FAR + 64), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(u=FAKE), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(u=2 * FAR), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(x_out=FAKE + 64), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(x_out=FAKE, x_out_stride=128), N.MOE_ERR_INVALID_ARG, "overlap"),
    (dict(gate=3 * FAR, gate_row=64, gate_col=1), N.MOE_ERR_INVALID_ARG, "overlap"),
])
def test_norm_refusals(kw, status, word):
    _refused(status, word, moe.moe_norm_residual, *_norm(**kw))


def test_norm_without_tokens_is_a_noop():
    moe.moe_norm_residual(*_norm(T=0, x=None, y=None, x_out=FAR))


def test_wrappers_name_what_is_wrong_with_a_tensor():
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.GroupedExperts(w)
    with pytest.raises(ValueError, match="order"):
        moe.GroupedExperts(w, order="out")
    with pytest.raises(ValueError, match="y_dtype"):
        moe.GroupedExperts(w, y_dtype=torch.int8)
    q, s = torch.zeros(2, 16, 16, dtype=torch.uint8), torch.zeros(2, 16, 1, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.W4Experts(q, s, group=32)
    with pytest.raises(ValueError, match="group"):
        moe.W4Experts(q, s, group=48)
    with pytest.raises(ValueError, match="x_dtype"):
        moe.W4Experts(q, s, group=32, x_dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.NormResidual(8, gamma_pre=torch.ones(8))
