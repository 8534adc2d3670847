"""The layer norm's gradient written over x, over the output's gradient and over the residual stream's: the bits of the call with
memory of its own, in all kernels."""
from __future__ import annotations

import pytest
import torch

from test_gpu_layer_norm import _CASES, _ID, _make, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", _CASES, ids=_ID)
def test_gradient_over_its_inputs(case):
    T, H, xt, yt, _, _, pad, _ = case
    gen, x, _, _, op = _make(case)
    dy, add = _rows(T, H, pad, yt, gen), _rows(T, H, pad, xt, gen)
    _, mean, rstd = op(x)

    def copy(t):
        return _rows(T, H, pad, t.dtype, gen).copy_(t)

    def run(over, add=None):
        at = {"x": x, "dy": dy, "add": add, "": x}
        mine = {n: copy(t) if n == over else t for n, t in at.items()}
        out = mine[over] if over else _rows(T, H, pad, xt, gen)
        sums = torch.full((H,), 7.0, device="cuda"), torch.full((H,), 7.0, device="cuda")
        dx, dg, db = op.backward(mine["dy"], mine["x"], mean, rstd, add=mine["add"], dx=out, dgamma=sums[0], dbeta=sums[1])
        assert dx is out
        if pad:                                            # what lies between the rows is left alone
            assert torch.isnan(dx.as_strided((T, pad), (H + pad, 1), dx.storage_offset() + H)).all()
        return dx, dg, db

    for a in (None, add):
        want = run("", a)
        for over in ("x",) + (("dy",) if xt is yt else ()) + (("add",) if a is not None else ()):
            assert all(torch.equal(g, w) for g, w in zip(run(over, a), want)), over
