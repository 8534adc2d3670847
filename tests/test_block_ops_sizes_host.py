"""Sizes beyond 32 bits are refused by the bindings of the dense product, layer norm and balance loss: cut off to 32 bits they would
be the sizes of a smaller call (no GPU)."""
from __future__ import annotations

import pytest

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

FAKE, FAR, BIG = 0x100000, 0x4000000000, 1 << 32           # nothing here is ever dereferenced


def _refused(word, fn, *args, **kw):
    with pytest.raises(N.MoeError, match=word) as ei:
        fn(*args, **kw)
    assert ei.value.status == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("T", [BIG, BIG + 1, 1 << 31, -BIG])
def test_rows_beyond_32_bits(T):
    plan = moe.moe_linear_plan_create(N.moe_linear_desc(N.MOE_BF16, N.MOE_F32, N.MOE_W_OUT_IN, 48, 64, FAKE, 64, None, N.MOE_F32,
                                                        N.MOE_ACT_NONE, 1.0, 1.0))
    try:
        _refused("T = ", moe.moe_linear_path, plan, T)
        _refused("T = ", moe.moe_linear, plan, FAKE, 64, T, None, N.MOE_F32, 0, FAR, 48, None, 0)
    finally:
        moe.moe_linear_plan_destroy(plan)
    norm = N.moe_layer_norm_desc(64, N.MOE_F32, N.MOE_F32, None, None, 1e-5)
    _refused("T = ", moe.moe_layer_norm, norm, FAKE, 64, T, FAR, 64, None, None, 0)
    _refused("T = ", moe.moe_layer_norm_backward_workspace_size, 64, T)
    _refused("T = ", moe.moe_layer_norm_backward, norm, FAKE, 64, FAR, 64, 2 * FAR, 3 * FAR, None, 0, T, 4 * FAR, 64, None, None, 0,
             None, 0, 0)
    balance = N.moe_balance_desc(N.MOE_ROUTE_SOFTMAX, 16, 2, 1.0, 0)
    _refused("T = ", moe.moe_balance_workspace_size, 16, T)
    _refused("n_seqs = ", moe.moe_balance_workspace_size, 16, 1, T)
    _refused("T = ", moe.moe_balance_loss, balance, FAKE, 16, FAR, T, None, 1, None, None, 2 * FAR, None, None, 0, None, 3 * FAR, 1 << 20, 0)
    _refused("n_seqs = ", moe.moe_balance_loss, balance, FAKE, 16, FAR, 8, 4 * FAR, T, None, None, 2 * FAR, None, None, 0, None, 3 * FAR,
             1 << 20, 0)


def test_descriptions_beyond_32_bits():
    _refused("n_in", N.moe_linear_desc, N.MOE_BF16, N.MOE_F32, N.MOE_W_OUT_IN, 48, BIG + 64)
    _refused("n_out", N.moe_linear_desc, n_out=BIG + 48)
    _refused("H = ", N.moe_layer_norm_desc, BIG + 64)
    _refused("top_k", N.moe_balance_desc, N.MOE_ROUTE_SOFTMAX, 16, BIG + 2)
    _refused("H = ", moe.moe_layer_norm_backward_workspace_size, BIG + 64, 1)
    _refused("n_experts", moe.moe_balance_workspace_size, BIG + 16, 1)
    _refused("n_experts", moe.BalanceLoss, BIG + 8, 2, device="cpu")
    assert N.moe_layer_norm_desc(64, eps=1e-6).H == 64
