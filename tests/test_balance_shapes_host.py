"""The balance loss's wrapper: ids and counts of the right number of entries in another order are refused, the same entries under
another shape are not; host tensors that report a device of their own, the library's calls recorded."""
from __future__ import annotations

import pytest
import torch

from test_block_ops_devices import _x, ops  # noqa: F401
from test_products_devices import _on

I32 = torch.int32


def _ids(*shape):
    return _on(torch.zeros(*shape, dtype=I32))


def test_ids_and_counts_in_another_order(ops):  # noqa: F811
    _, _, balance, calls, _ = ops                          # 8 experts, 2 a token; 4 tokens
    x, off = _x(width=8), _on(torch.zeros(4, dtype=I32))
    with pytest.raises(ValueError, match="ids must be"):
        balance(x, _ids(2, 4))
    with pytest.raises(ValueError, match="counts must be"):
        balance(x, _ids(4, 2), offsets=off, counts=_ids(8, 3))
    assert not calls
    for ids, kw in ((_ids(4, 2), {}), (_ids(8), {}), (_ids(2, 2, 2), {}), (_ids(4, 2), dict(offsets=off, counts=_ids(3, 8))),
                    (_ids(4, 2), dict(offsets=off, counts=_ids(24))), (_ids(4, 2), dict(counts=_ids(8, 1)))):
        balance(x, ids, **kw)
    assert len(calls) == 6
