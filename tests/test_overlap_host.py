"""Rows that share a byte are refused, in columns of one buffer as elsewhere (refusals only: no call gets to a launch)."""
from __future__ import annotations

import pytest

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N
from test_products_host import FAKE, FAR, _call, _dense, _norm, _refused


@pytest.mark.parametrize("kw", [
    dict(y=FAKE + 124, y_stride=256, x_stride=512),           # y begins in the last bytes of x's first row
    dict(y=FAKE + 1024 - 48 * 4 + 4, y_stride=256, x_stride=512),     # y's rows end in the next rows of x
    dict(y=FAKE + 3 * 1024 + 4, y_stride=256, x_stride=512),
    dict(y=FAKE - 2 * 1024 + 64, y_stride=256, x_stride=512),         # y begins two rows before x
    dict(y=FAKE + 512, y_stride=264, x_stride=512),           # columns of different strides drift into one another
])
def test_products_refuse_rows_that_share_a_byte(kw):
    plan = moe.moe_grouped_plan_create(_dense())
    try:
        _refused(N.MOE_ERR_INVALID_ARG, "overlaps", moe.moe_grouped_matmul, plan, *_call(**kw))
    finally:
        moe.moe_grouped_plan_destroy(plan)


@pytest.mark.parametrize("kw", [
    dict(x_out=FAR + 252, x_out_stride=128, y_stride=128),
    dict(x_out=FAR + 260, x_out_stride=128, y_stride=128),
    dict(x_out=3 * FAR, x_out_stride=96, u=3 * FAR + 252, u_stride=192),      # bf16 u beside fp32 x_out, one element in it
    dict(x_out=3 * FAR, x_out_stride=96, u=3 * FAR + 260, u_stride=192),      # and one past the row's end
    dict(gate=2 * FAR + 252, gate_row=128, gate_col=1, x_out_stride=128),
    dict(gate=2 * FAR + 256, gate_row=128, gate_col=2, x_out_stride=128),     # the gate's last column is the next row's first
])
def test_norm_refuses_rows_that_share_a_byte(kw):
    _refused(N.MOE_ERR_INVALID_ARG, "overlap", moe.moe_norm_residual, *_norm(**kw))
