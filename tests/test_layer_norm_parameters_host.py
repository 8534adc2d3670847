"""Layer norm's gamma and beta are read where they lie at each call: a parameter whose memory was replaced (moved, cast, laid into a
larger buffer) is not read at its old address; host tensors that report a device of their own, the library's calls recorded."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from test_block_ops_devices import _x, ops  # noqa: F401
from test_products_devices import _On, _on


def _calls(norm, calls):
    calls.clear()
    norm(_x())
    norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)))
    return [a[0] for _, a in calls]


@pytest.mark.parametrize("which", ["gamma", "beta"])
def test_replaced_memory_is_followed(ops, which):  # noqa: F811
    calls = ops[3]
    params = {n: _on(torch.ones(32)) for n in ("gamma", "beta")}
    norm = moe.LayerNorm(32, **params, y_dtype=torch.float32)
    for desc in _calls(norm, calls):
        assert (desc.gamma, desc.beta) == (params["gamma"].data_ptr(), params["beta"].data_ptr())
    old = params[which].data_ptr()
    keep = params[which].detach()                          # (so that the old address stays taken)
    new = torch.full((64,), 2.0)[8:40]
    params[which].data = new.as_subclass(_On)
    assert params[which].data_ptr() != old == keep.data_ptr()
    for desc in _calls(norm, calls):
        assert (desc.gamma, desc.beta) == (params["gamma"].data_ptr(), params["beta"].data_ptr())
    assert len(calls) == 2


@pytest.mark.parametrize("new", [torch.ones(32, dtype=torch.float16), torch.ones(31), torch.ones(64)[::2]])
def test_memory_that_no_longer_fits_is_refused(ops, new):  # noqa: F811
    calls = ops[3]
    gamma = _on(torch.ones(32))
    norm = moe.LayerNorm(32, gamma=gamma)
    norm(_x())
    keep = gamma.detach()
    gamma.data = new.as_subclass(_On)
    with pytest.raises(ValueError, match="gamma"):
        norm(_x())
    with pytest.raises(ValueError, match="gamma"):
        norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)))
    assert len(calls) == 1 and keep.numel() == 32
