"""The most rows of the dense product: refused beyond 2^30 by the call and by the question which kernel it runs (no GPU)."""
from __future__ import annotations

import pytest

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

FAKE = 0x100000                                            # nothing here is ever dereferenced


@pytest.fixture
def plan():
    p = moe.moe_linear_plan_create(N.moe_linear_desc(N.MOE_BF16, N.MOE_F32, N.MOE_W_OUT_IN, 48, 64, FAKE, 64, None, N.MOE_F32,
                                                     N.MOE_ACT_NONE, 1.0, 1.0))
    yield p
    moe.moe_linear_plan_destroy(p)


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 1])
def test_path_of_too_many_rows_is_refused(plan, T):
    with pytest.raises(N.MoeError, match="too large") as ei:
        moe.moe_linear_path(plan, T)
    assert ei.value.status == N.MOE_ERR_INVALID_ARG


def test_path_of_the_most_rows(plan):
    assert moe.moe_linear_path(plan, 1 << 30) == moe.moe_linear_path(plan, 1 << 24) == N.MOE_LINEAR_PAIRS
