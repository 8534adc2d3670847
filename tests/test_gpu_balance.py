"""The router's balance loss, counts and gradient on the GPU against the definition in 64 bits.

Tolerance, before any run; u = 2^-24, R: the largest distance of a logit from its token's largest that is not -inf.  l - max is
off by u R, its exponential by 2 units more; sums over a token's experts (at most 32 in a lane, a tree of 5) by 40 u: p is off by
at most (R + 48) u relative (sigmoid: e^-|l|, the division and 1 - s a few units more: (R + 60) u).  With f' = f - 1 the
gradient is a p (f' - sum f' p): off by a p u (R + 60) (|f'| + 2 sum |f'| p) + roundings u a p (...) and its own p's error:
a p u (2 R + 130) (|f'| + sum |f'| p) in all.  The loss is a sum of positive terms: p's error, at most T / 16 + 80
additions one after another: (R + 130 + T / 16) u.  Counts are exact.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


def _inputs(T, E, k, seed=0, pad=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(T * 3 + E + seed)
    full = torch.full((T, E + pad), float("nan"), device="cuda")
    full[:, :E] = spread * torch.randn(T, E, generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")
    logits = full[:, :E]
    ids = torch.topk(logits, k, dim=1).indices.sort(1).values.int().contiguous() if T else torch.zeros(0, k, dtype=torch.int32, device="cuda")
    return logits, ids


def _want(logits, ids, k, mode, coef, off=None, mask=None):
    """(loss, counts, dlogits, tolerance of the loss, of dlogits); p and f of each token by the definition."""
    T, E = logits.shape
    off = [0, T] if off is None else list(off)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    rows = [a + keep[a:b].nonzero()[:, 0] for a, b in zip(off[:-1], off[1:])]
    used = sum(len(r) > 0 for r in rows)
    counts = torch.zeros(len(rows), E, dtype=torch.int32, device="cuda")
    grad, tol = torch.zeros(T, E, dtype=torch.float64, device="cuda"), torch.zeros(T, E, dtype=torch.float64, device="cuda")
    loss, R = 0.0, 0.0
    for b, r in enumerate(rows):
        if not len(r):
            continue
        v = logits[r].double()
        top = v.amax(1, keepdim=True)
        fin = torch.where(v > -INF, top - v, torch.zeros_like(v))
        R = max(R, float(fin.nan_to_num(0.0).max()))
        if mode == "softmax":
            s, slope = torch.where(v > -INF, torch.exp(v - top), torch.zeros_like(v)), 1.0
        else:
            # (relative to the largest, as sigmoid alone underflows for a token of very low logits)
            s = torch.where(v > -INF, torch.exp(v.clamp(max=0) - top.clamp(max=0)) * torch.sigmoid(v.abs()), torch.zeros_like(v))
            s = torch.where(v > 0, torch.sigmoid(v), s)
            slope = torch.sigmoid(-v)
        tot = s.sum(1, keepdim=True)
        p = s / torch.where(tot > 0, tot, torch.ones_like(tot))
        counts[b] = torch.bincount(ids[r].reshape(-1).long(), minlength=E)
        f = counts[b].double() * E / (k * len(r))
        a = coef / (used * len(r))
        loss += a * float((f * p).sum())
        grad[r] = a * p * (f - (p @ f)[:, None]) * slope
        f1 = (f - 1).abs()
        tol[r] = a * p * U * (2 * R + 130) * (f1 + (p @ f1)[:, None])
    return loss, counts, grad, (R + 130 + T / 16) * U * abs(loss), tol


def _compare(got, want, upstream=1.0, base=None):
    loss, counts, dlogits = got
    w_loss, w_counts, w_grad, t_loss, t_grad = want
    assert torch.equal(counts, w_counts)
    assert abs(loss.item() - w_loss) <= t_loss + U * abs(w_loss)
    if dlogits is not None:
        w, t = upstream * w_grad, abs(upstream) * t_grad
        if base is not None:
            w, t = w + base.double(), t + U * (base.double() + w).abs()
        bad = (dlogits.double() - w).abs() - (t + U * w.abs() + 2.0 ** -149)
        assert (bad <= 0).all(), (bad.max(), int((bad > 0).sum()))


_SIZES = [(1, 1, 1, 0), (1, 8, 2, 0), (3, 7, 3, 0), (32, 128, 8, 0), (33, 31, 4, 1), (100, 33, 1, 0), (64, 256, 8, 0), (65, 256, 8, 0), (257, 130, 8, 4), (1000, 256, 8, 0),
          (4096, 128, 8, 0), (700, 255, 5, 3), (77, 500, 6, 0), (130, 512, 8, 4), (40, 1024, 32, 0), (50, 1001, 7, 0), (9000, 64, 6, 0)]


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k, pad", _SIZES)
def test_balance(T, E, k, pad, mode):
    logits, ids = _inputs(T, E, k, pad=pad)
    op = moe.BalanceLoss(E, k, mode=mode, coef=0.5)
    want = _want(logits, ids, k, mode, 0.5)
    got = op(logits, ids, dlogits=True)
    _compare(got, want)
    loss, counts, none = op(logits, ids)
    assert none is None and torch.equal(loss, got[0]) and torch.equal(counts, got[1])
    # an upstream gradient, rows of another stride, added to what is there, in place
    up = torch.tensor([-3.0], device="cuda")
    buf = torch.randn(T, E + 5, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    d, base = buf[:, :E], buf.clone()
    out = op(logits, ids, dlogits=d, upstream=up, accumulate=True)
    _compare(out, want, -3.0, base[:, :E])
    assert torch.equal(buf[:, E:], base[:, E:])
    same = logits.clone()
    _, _, d2 = op(same, ids, dlogits=same)
    assert d2 is same and torch.equal(same, got[2])
    assert op.device_status() == N.MOE_OK


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k, off", [
    (100, 32, 4, [0, 100]), (100, 32, 4, [3, 50, 90]), (100, 33, 4, [0, 0, 1, 1, 60, 100, 100]), (5, 8, 2, [5, 5]), (64, 128, 8, [0, 0, 0]),
    (5000, 128, 8, [0, 1, 17, 1000, 1000, 4200, 4999]), (3000, 256, 8, list(range(0, 2990, 13))), (40, 16, 2, list(range(41))),
])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_of_sequences(T, E, k, off, mode, masked):
    logits, ids = _inputs(T, E, k, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(T)
    mask = torch.rand(T, device="cuda", generator=gen) < 0.7 if masked else None
    if masked:
        mask[off[0]: off[1]] = False                       # a sequence of which nothing counts
        bad = torch.where(mask, 0, 1).bool()
        logits[bad] = float("nan")                         # what a padded place holds does not matter
        ids[bad] = 10 ** 6
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    op = moe.BalanceLoss(E, k, mode=mode, coef=2.0)
    want = _want(logits, ids, k, mode, 2.0, off, mask)
    got = op(logits, ids, offsets=o, mask=mask, dlogits=True)
    _compare(got, want)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[off[0]: off[-1]] = False
    if masked:
        outside |= ~mask
    assert bool((got[2][outside] == 0).all())
    d = torch.full((T, E), 7.0, device="cuda")
    op(logits, ids, offsets=o, mask=mask.to(torch.uint8) if masked else None, dlogits=d, accumulate=True)
    assert bool((d[outside] == 7.0).all())
    assert op.device_status() == N.MOE_OK


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k, off, live", [
    (100000, 300, 2, [0, 100000], None), (100000, 300, 2, [7, 60000, 99990], None),      # more steps a warp than bits of a word
    (20000, 64, 8, [0, 15000, 20000], [(14990, 15000), (15001, 15002)]),                 # what counts lies many chunks behind the start
    (20000, 64, 8, [0, 9000, 9000, 20000], [(9000, 20000)]), (20000, 64, 8, [0, 20000], [(19999, 20000)]),
    (20000, 64, 8, [0, 10000, 20000], [(0, 1), (5000, 9000), (19999, 20000)]), (20000, 64, 8, [0, 20000], []),
    (64, 256, 8, [0, 30, 64], [(0, 10), (50, 64)]), (64, 260, 8, [0, 30, 64], [(0, 10), (50, 64)]), (64, 128, 8, [0, 30, 60, 64], [(31, 64)]),
])
def test_balance_of_masked_stretches(T, E, k, off, live, mode):
    logits, ids = _inputs(T, E, k, seed=4)
    if live is None:
        mask = torch.rand(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)) < 0.5
    else:
        mask = torch.zeros(T, dtype=torch.bool, device="cuda")
        for a, b in live:
            mask[a:b] = True
    logits[~mask] = float("nan")
    op = moe.BalanceLoss(E, k, mode=mode)
    got = op(logits, ids, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), mask=mask, dlogits=True)
    _compare(got, _want(logits, ids, k, mode, 1.0, off, mask))
    assert bool((got[2][~mask] == 0).all()) and op.device_status() == N.MOE_OK


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_balance_of_far_logits_and_infinities(mode):
    T, E, k = 64, 40, 4
    logits, ids = _inputs(T, E, k, seed=2, spread=30.0)
    logits[5] = -INF                                       # a token without a probability
    logits[6, 3:] = -INF
    logits[7] -= 500.0                                     # sigmoid underflows, its shares do not
    logits[8] += 500.0
    logits[9] = torch.finfo(torch.float32).min             # a mask of the lowest value: all alike
    logits[10, ::2] = torch.finfo(torch.float32).min
    op = moe.BalanceLoss(E, k, mode=mode)
    got = op(logits, ids, dlogits=True)
    # (row 10's distance would be the tolerance's R: the lowest values' p are 0 on both sides, so leave them out of R)
    seen = logits.clone()
    seen[10, ::2] = -INF
    _compare(got, _want(seen, ids, k, mode, 1.0))
    assert bool((got[2][5] == 0).all())
    bad = logits.clone()
    bad[11, 7], bad[12, 7] = float("nan"), INF
    _, _, d = op(bad, ids, dlogits=True)
    rows = [i for i in range(T) if i not in (11, 12)]
    assert torch.equal(d[rows], got[2][rows]) and torch.isnan(d[11]).all()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(mode):
    """Central differences of the definition in 64 bits with the counts held: off by 1e-8 of derivatives of order 1."""
    T, E, k = 20, 24, 3
    logits, ids = _inputs(T, E, k, seed=3)
    off = [0, 7, 20]
    op = moe.BalanceLoss(E, k, mode=mode)
    _, counts, d = op(logits, ids, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dlogits=True)

    def loss(v):
        s = torch.softmax(v, 1) if mode == "softmax" else torch.sigmoid(v)
        p = s / s.sum(1, keepdim=True)
        return sum((counts[b].double() * E / (k * (z - a) ** 2) * p[a:z]).sum() / 2 for b, (a, z) in enumerate(zip(off, off[1:])))

    gen = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        v = torch.randn(T, E, generator=gen, device="cuda").double()
        diff = (loss(logits.double() + 1e-4 * v) - loss(logits.double() - 1e-4 * v)) / 2e-4
        assert abs(diff - (d.double() * v).sum()) <= 1e-5 * (d.double() * v).norm() + 1e-8


def test_balance_even_load_has_no_gradient():
    T, E, k = 64, 16, 2
    logits, _ = _inputs(T, E, k)
    ids = ((torch.arange(T, device="cuda")[:, None] * k + torch.arange(k, device="cuda")) % E).int()
    loss, counts, d = moe.BalanceLoss(E, k)(logits, ids, dlogits=True)
    assert bool((counts == T * k // E).all()) and abs(loss.item() - 1) < 1e-6 and bool((d == 0).all())


def test_balance_bad_ids_and_offsets_are_reported():
    T, E, k = 50, 16, 2
    logits, ids = _inputs(T, E, k)
    op, other = moe.BalanceLoss(E, k), moe.BalanceLoss(E, k)
    bad = ids.clone()
    bad[3, 1], bad[9, 0] = E, -1
    _, counts, _ = op(logits, bad)
    assert op.device_status(clear=True) == N.MOE_ERR_DEVICE_CHECK and int(counts.sum()) == T * k - 2
    for off in ([0, T + 1], [-1, 5], [0, 30, 20, T]):
        op(logits, ids, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dlogits=True)
        assert op.device_status(clear=True) == N.MOE_ERR_DEVICE_CHECK
    assert other.device_status() == N.MOE_OK
    _compare(op(logits, ids, dlogits=True), _want(logits, ids, k, "softmax", 1.0))


def test_balance_without_tokens():
    op = moe.BalanceLoss(8, 2)
    logits, ids = _inputs(0, 8, 2)
    loss, counts, d = op(logits, ids, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"), dlogits=True)
    assert loss.item() == 0 and counts.shape == (3, 8) and bool((counts == 0).all()) and d.shape == (0, 8)


@pytest.mark.parametrize("T, E", [(32, 128), (5000, 64)])
def test_balance_captured_two_at_once_and_on_another_stream(T, E):
    k = 4
    logits, ids = _inputs(T, E, k)
    op = moe.BalanceLoss(E, k)
    ref = [t.clone() for t in op(logits, ids, dlogits=True)]
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            outs.append(op(logits, ids, dlogits=True))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = op(logits, ids, dlogits=True, stream=streams[2])
        torch.cuda.synchronize()
        for got in outs + [eager]:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_balance_of_rows_that_lie_far_apart():
    """Strides of 2^30 + 4 elements: offsets beyond 32 bits in elements and bytes."""
    T, E, k, far = 5, 64, 4, (1 << 30) + 4
    logits, ids = _inputs(T, E, k)
    op = moe.BalanceLoss(E, k)
    want = op(logits, ids, dlogits=True)
    buf = torch.empty(4 * far + 2 * E, device="cuda")
    l, d = (buf[i * E:].as_strided((T, E), (far, 1)) for i in range(2))
    l.copy_(logits)
    got = op(l, ids, dlogits=d)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
