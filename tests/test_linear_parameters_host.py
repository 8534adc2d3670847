"""A dense product whose weights or bias have been laid elsewhere since it was made is refused: its plan holds the old address.  Host
tensors that report a device of their own, the library's calls recorded."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from test_block_ops_devices import _x, ops  # noqa: F401
from test_products_devices import _On, _on

BF = torch.bfloat16


@pytest.mark.parametrize("which", ["w", "bias"])
def test_replaced_memory_is_refused(ops, which):  # noqa: F811
    calls = ops[3]
    params = dict(w=_on(torch.zeros(16, 32, dtype=BF)), bias=_on(torch.zeros(16)))
    op = moe.Linear(**params)
    op(_x(BF))
    params[which].fill_(2.0)                               # written in place: fine
    op(_x(BF))
    assert len(calls) == 2
    keep = params[which].detach()                          # (so that the old address stays taken)
    params[which].data = torch.zeros_like(keep).as_subclass(_On)
    with pytest.raises(ValueError, match="replaced"):
        op(_x(BF))
    assert len(calls) == 2 and keep.numel()
