"""An upstream gradient of the balance loss that is not finite (a loss scale that overflowed) stays in the rows that it
belongs to: tokens that do not count and tokens without a probability have a gradient of exactly 0."""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

INF = float("inf")
# T, E, k, offsets: one launch and two, read four logits at a time and one by one, several tokens a warp and one; no
# token that counts (of 130)
_CASES = [(20, 32, 4, None), (20, 33, 4, [0, 12, 18]), (300, 40, 4, None), (300, 39, 3, [2, 100, 100, 290]), (700, 256, 8, [0, 300, 700]),
          (130, 512, 8, [0, 130]), (90, 1001, 5, [0, 40, 90])]


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
@pytest.mark.parametrize("T, E, k, off", _CASES)
def test_rows_without_a_gradient_stay_zero(T, E, k, off, mode, value):
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices.int()
    mask = torch.rand(T, device="cuda", generator=gen) < 0.6
    mask[-10:] = True
    nothing = torch.zeros(T, dtype=torch.bool, device="cuda")
    nothing[T // 2] = nothing[T - 12] = True
    logits[nothing] = -INF
    if off is not None:
        mask[off[0]: off[1]] = False                       # a sequence of which nothing counts
    counted = mask & ~nothing
    if off is not None:
        counted[: off[0]] = False
        counted[off[-1]:] = False
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    op = moe.BalanceLoss(E, k, mode=mode)
    up = torch.full((1,), value, device="cuda")
    loss, _, ref = op(logits, ids, offsets=o, mask=mask, dlogits=True)
    got_loss, _, got = op(logits, ids, offsets=o, mask=mask, dlogits=True, upstream=up)
    assert torch.equal(loss, got_loss) and bool(counted.any()) == (off is None or len(off) > 2) and not bool(counted.all())
    assert bool((got[~counted] == 0).all())
    assert not bool(torch.isfinite(got[counted][ref[counted] != 0]).any())
    base = torch.randn(T, E, generator=gen, device="cuda")
    d = base.clone()
    op(logits, ids, offsets=o, mask=mask, dlogits=d, upstream=up, accumulate=True)
    assert torch.equal(d[~counted], base[~counted])
