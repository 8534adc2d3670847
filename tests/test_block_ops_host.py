"""Refusals of the dense product, layer norm and balance loss calls: named on the host, before any launch (no GPU)."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

FAKE = 0x100000
FAR = 0x4000000000          # addresses far from one another: nothing here is ever dereferenced
BAD, UNS, WS = N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_WORKSPACE


def _refused(status, word, fn, *args):
    with pytest.raises(N.MoeError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)
    assert word in str(ei.value), str(ei.value)


def _with(defaults, kw):
    assert set(kw) <= set(defaults), kw
    return list({**defaults, **kw}.values())


_PLAN = dict(type=N.MOE_BF16, y_type=N.MOE_F32, order=N.MOE_W_OUT_IN, n_out=48, n_in=64, w=FAKE, row_stride=64, bias=None,
             bias_type=N.MOE_F32, act=N.MOE_ACT_NONE, scale=1.0, res_scale=1.0)


@pytest.mark.parametrize("kw, status, word", [
    (dict(type=N.MOE_F32), UNS, "type"), (dict(y_type=N.MOE_Q8_0), UNS, "y_type"), (dict(order=2), BAD, "order"),
    (dict(n_out=0), BAD, "n_out"), (dict(n_in=(1 << 20) + 1, row_stride=(1 << 20) + 8), BAD, "n_in"), (dict(w=None), BAD, "NULL"),
    (dict(w=FAKE + 8), BAD, "aligned"), (dict(row_stride=56), BAD, "row_stride"), (dict(row_stride=68), BAD, "row_stride"),
    (dict(order=N.MOE_W_IN_OUT, row_stride=40), BAD, "row_stride"), (dict(bias=FAKE, bias_type=N.MOE_Q4_K), UNS, "bias_type"),
    (dict(bias=FAKE + 2), BAD, "bias"), (dict(act=5), UNS, "act"), (dict(act=-1), UNS, "act"),
    (dict(scale=float("inf")), BAD, "scale"), (dict(res_scale=float("nan")), BAD, "scale"),
])
def test_linear_plan_refusals(kw, status, word):
    _refused(status, word, moe.moe_linear_plan_create, N.moe_linear_desc(*_with(_PLAN, kw)))


_LINEAR = dict(x=FAKE, x_stride=64, T=3, r=2 * FAR, r_type=N.MOE_F32, r_stride=48, y=FAR, y_stride=48, status=None, stream=0)


@pytest.mark.parametrize("kw, status, word", [
    (dict(T=-1), BAD, "T = -1"), (dict(T=(1 << 30) + 1), BAD, "too large"), (dict(x=None), BAD, "NULL"), (dict(y=None), BAD, "NULL"),
    (dict(r_type=N.MOE_Q8_0), UNS, "r_type"), (dict(x=FAKE + 8), BAD, "aligned"), (dict(y=FAR + 2), BAD, "aligned"),
    (dict(r=FAR + 2), BAD, "aligned"), (dict(status=FAKE + 1), BAD, "aligned"), (dict(x_stride=56), BAD, "x_stride"),
    (dict(x_stride=68), BAD, "x_stride"), (dict(y_stride=47), BAD, "y_stride"), (dict(r_stride=47), BAD, "r_stride"),
    (dict(y_stride=(1 << 32) + 1), BAD, "y_stride"), (dict(y=FAKE + 256), BAD, "overlaps x"), (dict(r=FAR + 192), BAD, "overlaps r"),
    (dict(r=FAR, r_stride=64), BAD, "overlaps r"), (dict(r=FAR, r_type=N.MOE_BF16), BAD, "overlaps r"),
    (dict(x=3 * FAR, y=FAKE + 48 * 128 - 4), BAD, "overlaps w"), (dict(status=FAR + 3 * 192 - 4), BAD, "status overlaps"),
    (dict(status=FAKE + 8), BAD, "status overlaps"), (dict(status=2 * FAR), BAD, "status overlaps"),
])
def test_linear_call_refusals(kw, status, word):
    plan = moe.moe_linear_plan_create(N.moe_linear_desc(*_PLAN.values()))
    try:
        _refused(status, word, moe.moe_linear, plan, *_with(_LINEAR, kw))
        moe.moe_linear(plan, *_with(_LINEAR, dict(T=0, x=None, y=None)))       # no rows: nothing launched
        assert moe.moe_linear_path(plan, 1) == N.MOE_LINEAR_SPLIT
        _refused(BAD, "T = 0", moe.moe_linear_path, plan, 0)
    finally:
        moe.moe_linear_plan_destroy(plan)
    _refused(BAD, "plan", moe.moe_linear, None, *_LINEAR.values())


def test_linear_path_by_size():
    plan = moe.moe_linear_plan_create(N.moe_linear_desc(*_with(_PLAN, dict(n_out=7168, n_in=2048, row_stride=2048))))
    try:
        assert moe.moe_linear_path(plan, 1) == moe.moe_linear_path(plan, 64) == N.MOE_LINEAR_SPLIT
        assert moe.moe_linear_path(plan, 4096) == N.MOE_LINEAR_PAIRS
    finally:
        moe.moe_linear_plan_destroy(plan)


_NORM = dict(H=64, x_type=N.MOE_F32, y_type=N.MOE_F32, gamma=FAKE, beta=FAKE, eps=1e-5)
_FORWARD = dict(x=FAR, x_stride=64, T=4, y=2 * FAR, y_stride=64, mean=3 * FAR, rstd=4 * FAR, stream=0)
_BACKWARD = dict(dy=FAR, dy_stride=64, x=2 * FAR, x_stride=64, mean=3 * FAR, rstd=4 * FAR, add=5 * FAR, add_stride=64, T=4, dx=6 * FAR,
                 dx_stride=64, dgamma=7 * FAR, dbeta=8 * FAR, accumulate=0, workspace=9 * FAR, ws_bytes=1 << 20, stream=0)
_DESC = [(dict(H=0), BAD, "H = 0"), (dict(H=32769), BAD, "H = 32769"), (dict(x_type=N.MOE_Q8_0), UNS, "types"),
         (dict(y_type=N.MOE_Q4_K), UNS, "types"), (dict(eps=-1e-6), BAD, "eps"), (dict(eps=float("nan")), BAD, "eps"),
         (dict(gamma=FAKE + 2), BAD, "aligned"), (dict(T=-2), BAD, "T = -2"), (dict(T=(1 << 30) + 1), BAD, "too large")]


def _split(call, kw):
    return ([N.moe_layer_norm_desc(*_with(_NORM, {n: v for n, v in kw.items() if n in _NORM}))]
            + _with(call, {n: v for n, v in kw.items() if n not in _NORM}))


@pytest.mark.parametrize("kw, status, word", _DESC + [
    (dict(x=None), BAD, "NULL"), (dict(y=None, mean=None, rstd=None), BAD, "none"), (dict(x_stride=63), BAD, "stride"),
    (dict(y_stride=-64), BAD, "stride"), (dict(x=FAR + 2), BAD, "aligned"), (dict(mean=FAR + 1), BAD, "aligned"),
    (dict(y=FAR + 64), BAD, "overlap"), (dict(y=FAR, y_stride=128), BAD, "overlap"), (dict(mean=FAR), BAD, "overlap"),
    (dict(rstd=3 * FAR + 4), BAD, "overlap"), (dict(y=FAKE), BAD, "overlap"), (dict(mean=FAKE + 8), BAD, "overlap"),
    (dict(y=FAR, y_type=N.MOE_BF16), BAD, "overlap"),
])
def test_layer_norm_refusals(kw, status, word):
    _refused(status, word, moe.moe_layer_norm, *_split(_FORWARD, kw))


@pytest.mark.parametrize("kw, status, word", _DESC + [
    (dict(x=None), BAD, "NULL"), (dict(dy=None), BAD, "NULL"), (dict(mean=None), BAD, "NULL"), (dict(rstd=None), BAD, "NULL"),
    (dict(dx=None, dgamma=None, dbeta=None), BAD, "none"), (dict(add_stride=63), BAD, "stride"), (dict(dx_stride=0), BAD, "stride"),
    (dict(dy=FAR + 2), BAD, "aligned"), (dict(dgamma=FAR + 2), BAD, "aligned"), (dict(workspace=None), WS, "workspace"),
    (dict(ws_bytes=4 * 2 * 64 * 4 - 1), WS, "workspace"), (dict(workspace=9 * FAR + 128), BAD, "aligned"),
    (dict(dx=FAR + 64), BAD, "overlap"), (dict(dx=2 * FAR, dx_stride=128), BAD, "overlap"), (dict(dx=3 * FAR), BAD, "overlap"),
    (dict(dgamma=8 * FAR), BAD, "overlap"), (dict(dgamma=FAR), BAD, "overlap"), (dict(dbeta=FAKE), BAD, "overlap"),
    (dict(workspace=6 * FAR), BAD, "overlap"), (dict(workspace=7 * FAR), BAD, "overlap"), (dict(dx=FAR, y_type=N.MOE_BF16), BAD, "overlap"),
])
def test_layer_norm_backward_refusals(kw, status, word):
    _refused(status, word, moe.moe_layer_norm_backward, *_split(_BACKWARD, kw))


def test_layer_norm_without_rows_is_a_noop():
    moe.moe_layer_norm(*_split(_FORWARD, dict(T=0, x=None)))
    moe.moe_layer_norm_backward(*_split(_BACKWARD, dict(T=0, x=None, dy=None, dgamma=None, dbeta=None, workspace=None)))
    moe.moe_layer_norm_backward(*_split(_BACKWARD, dict(T=0, x=None, dy=None, accumulate=1, workspace=None)))
    assert moe.moe_layer_norm_backward_workspace_size(64, 0) == 0 < moe.moe_layer_norm_backward_workspace_size(64, 1)
    assert moe.moe_layer_norm_backward_workspace_size(64, 1 << 30) == moe.moe_layer_norm_backward_workspace_size(64, 1 << 20)
    _refused(BAD, "H = 0", moe.moe_layer_norm_backward_workspace_size, 0, 1)


_BAL = dict(mode=N.MOE_ROUTE_SOFTMAX, n_experts=16, top_k=2, coef=1.0, accumulate=0)
_BALANCE = dict(logits=FAR, stride=16, ids=2 * FAR, T=10, seq_offsets=3 * FAR, n_seqs=2, mask=4 * FAR, upstream=5 * FAR, loss=6 * FAR,
                counts=7 * FAR, dlogits=8 * FAR, dstride=16, status=9 * FAR, workspace=10 * FAR, ws_bytes=1 << 20, stream=0)


def _balance(kw):
    return ([N.moe_balance_desc(*_with(_BAL, {n: v for n, v in kw.items() if n in _BAL}))]
            + _with(_BALANCE, {n: v for n, v in kw.items() if n not in _BAL}))


@pytest.mark.parametrize("kw, status, word", [
    (dict(mode=2), BAD, "mode"), (dict(n_experts=0), BAD, "n_experts"), (dict(n_experts=1025), BAD, "n_experts"), (dict(top_k=0), BAD, "top_k"),
    (dict(top_k=17), BAD, "top_k"), (dict(n_experts=64, top_k=33, stride=64, dstride=64), BAD, "top_k"),
    (dict(coef=float("nan")), BAD, "coef"), (dict(T=-1), BAD, "T = -1"), (dict(T=1 << 30), BAD, "too large"),
    (dict(n_seqs=0), BAD, "n_seqs"), (dict(n_seqs=65536), BAD, "n_seqs"), (dict(seq_offsets=None), BAD, "seq_offsets"),
    (dict(loss=None, counts=None, dlogits=None), BAD, "none"), (dict(logits=None), BAD, "NULL"), (dict(ids=None), BAD, "NULL"),
    (dict(logits=FAR + 2), BAD, "aligned"), (dict(ids=FAR + 1), BAD, "aligned"), (dict(counts=FAR + 2), BAD, "aligned"),
    (dict(stride=15), BAD, "stride"), (dict(dstride=15), BAD, "stride"), (dict(workspace=None), WS, "workspace"),
    (dict(ws_bytes=100), WS, "workspace"), (dict(workspace=10 * FAR + 16), BAD, "aligned"),
    (dict(dlogits=FAR, accumulate=1), BAD, "nothing to add"), (dict(dlogits=FAR + 64), BAD, "overlaps"),
    (dict(dlogits=FAR, dstride=32), BAD, "overlaps"), (dict(loss=FAR + 4), BAD, "overlaps"), (dict(counts=2 * FAR + 8), BAD, "overlaps"),
    (dict(loss=7 * FAR), BAD, "overlaps"), (dict(status=8 * FAR), BAD, "overlaps"), (dict(workspace=8 * FAR), BAD, "overlaps"),
    (dict(dlogits=4 * FAR), BAD, "overlaps"), (dict(loss=5 * FAR), BAD, "overlaps"),
])
def test_balance_refusals(kw, status, word):
    _refused(status, word, moe.moe_balance_loss, *_balance(kw))


def test_balance_workspace_size():
    assert moe.moe_balance_workspace_size(16, 0) > 0
    assert moe.moe_balance_workspace_size(16, 1 << 20, 100) > moe.moe_balance_workspace_size(16, 1 << 20)
    _refused(BAD, "n_seqs", moe.moe_balance_workspace_size, 16, 1, 0)


def test_wrappers_name_what_is_wrong_with_a_tensor():
    w = torch.zeros(16, 32, dtype=torch.bfloat16)
    for kw, word in ((dict(), "CUDA"), (dict(order="out"), "order"), (dict(act="tanh"), "act"), (dict(y_dtype=torch.int8), "y_dtype")):
        with pytest.raises(ValueError, match=word):
            moe.Linear(w, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        moe.LayerNorm(8, gamma=torch.ones(8))
    with pytest.raises(ValueError, match="y_dtype"):
        moe.LayerNorm(8, y_dtype=torch.int8)
    with pytest.raises(ValueError, match="x must be"):
        moe.LayerNorm(8)(torch.zeros(2, 8))
    with pytest.raises(ValueError, match="mode"):
        moe.BalanceLoss(8, 2, mode="tanh")
    op = moe.BalanceLoss(8, 2, device="cpu")
    with pytest.raises(ValueError, match="logits"):
        op(torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32))
