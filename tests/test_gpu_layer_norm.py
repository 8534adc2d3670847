"""Layer norm and its gradient on the GPU against the formulas in 64 bits, and the gradient against differences.

Tolerance, before any run; u = 2^-24.  A thread adds at most 32 elements of a row one after another, the rest is a tree of at
most 11 levels: a sum over the row is off by at most 44 u times the sum of absolute values.  The mean m that is
taken off first is off by that much, but the rest d of it is found and taken off as well: what is left is the
error of d, at most 44 u mean |x - m| <= 44 u s (s: the row's deviation), and the rounding of x - m.  So
  |xh error| <= 48 u + 4 u |xh| + |xh| (half of the variance's 46 u, and 3 roundings) <= u (48 + 32 |xh|) =: e,
y = xh gamma + beta adds 2 roundings; mean: u |m| + 46 u s; rstd: 30 u relative.
Backward: mean g and mean g xh are off by 44 u mean |g| and 44 u mean |g xh| + mean |g e|; dx = add + q (g - mean g - xh mean(g xh)):
  q (44 u (mean |g| + |xh| mean |g xh|) + |xh| mean |g e| + e |mean g xh| + 4 u (|g| + |mean g| + |xh mean g xh|)) + u (|add| + |dx|).
A sum over the rows: rows one after another in a group (at most T / 150 + 1), then at most 16 groups and 32 + 16 partial sums:
u (T / 150 + 66) times the sum of absolute values, and the errors of xh.  Storing adds half a step of the output's type.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def _rows(T, H, pad, dtype, gen, scale=1.0, at=0.0):
    full = torch.full((T, H + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :H] = torch.randn(T, H, generator=gen, device="cuda") * scale + at
    return full[:, :H]


def _close(got, want, tol):
    t = got.dtype
    tol = tol + torch.finfo(t).eps / 2 * (want.abs() + tol) + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    bad = (got.double() - want).abs() - tol
    assert (bad <= 0).all(), (bad.max(), int((bad > 0).sum()))


def _stats(x, eps):
    m = x.double().mean(1, keepdim=True)
    q = 1 / ((x.double() - m).pow(2).mean(1, keepdim=True) + eps).sqrt()
    xh = (x.double() - m) * q
    return m, q, xh, U * (48 + 32 * xh.abs())


_CASES = [
    # T, H, x type, y type, gamma, beta, pad, mean / deviation
    (1, 1, F32, F32, True, True, 0, 0), (1, 2048, F32, BF, True, True, 0, 0), (3, 7, BF, F32, True, False, 0, 0),
    (5, 64, F32, BF, False, True, 0, 1), (19, 256, HF, HF, True, True, 8, 0), (70, 264, BF, BF, True, True, 8, 0),
    (9, 512, F32, F32, True, True, 0, 1000), (7, 768, BF, F32, False, False, 0, 0), (4, 1024, F32, BF, True, True, 4, 30),
    (5, 1023, F32, F32, True, True, 0, 30), (33, 1000, F32, BF, True, True, 3, 0), (4, 2047, BF, BF, True, True, 1, 0),
    (300, 2048, F32, BF, True, True, 0, 1000), (6, 4096, F32, F32, True, True, 0, 0), (6, 4095, HF, F32, True, True, 0, 0),
    (40, 7168, BF, BF, True, True, 8, 0), (3, 7169, F32, BF, True, True, 0, 0), (1000, 100, BF, HF, True, True, 0, 0),
    (2, 8192, F32, F32, True, True, 0, 1), (3, 8200, BF, BF, True, True, 0, 1), (2, 16384, F32, BF, True, True, 0, 0),
    (2, 16383, BF, BF, True, False, 0, 0), (2, 32768, F32, F32, True, True, 0, 100), (2, 32767, F32, HF, False, True, 5, 0),
    (2500, 8200, BF, BF, True, True, 0, 0),
    # more rows than two for each SM: the kernels by type, rows of all their channels and not, read 16 bytes, 8 bytes and one by one
    (400, 512, F32, F32, True, True, 0, 100), (400, 1000, F32, BF, True, True, 0, 1), (400, 2048, F32, HF, True, True, 4, 1),
    (400, 4096, BF, BF, True, True, 0, 1), (400, 1024, HF, HF, True, True, 8, 0), (400, 1004, BF, BF, True, True, 0, 1),
    (400, 1024, BF, F32, True, True, 0, 1), (400, 777, HF, F32, True, False, 0, 1), (400, 777, BF, BF, False, True, 3, 1),
    (400, 64, F32, BF, True, True, 1, 1), (400, 8192, F32, F32, True, True, 0, 1), (400, 8184, BF, BF, True, True, 0, 1),
    (400, 7168, HF, HF, True, True, 8, 0), (400, 3, F32, F32, True, True, 0, 0), (400, 600, HF, BF, True, True, 0, 1),
    (4000, 320, F32, BF, True, True, 0, 1), (9000, 40, BF, BF, True, True, 0, 1),
]
_ID = lambda c: "-".join(str(v).replace("torch.", "") for v in c)  # noqa: E731


def _make(case):
    T, H, xt, yt, g, b, pad, at = case
    gen = torch.Generator(device="cuda").manual_seed(H * 7 + T)
    x = _rows(T, H, pad, xt, gen, 2.0, 2.0 * at)
    gamma = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda") if g else None
    beta = torch.randn(H, generator=gen, device="cuda") if b else None
    return gen, x, gamma, beta, moe.LayerNorm(H, gamma=gamma, beta=beta, eps=1e-5, y_dtype=yt)


@pytest.mark.parametrize("case", _CASES, ids=_ID)
def test_layer_norm(case):
    T, H, xt, yt, _, _, pad, _ = case
    gen, x, gamma, beta, op = _make(case)
    out = _rows(T, H, pad, yt, gen)
    y, mean, rstd = op(x, out=out)
    assert y is out
    m, q, xh, e = _stats(x, 1e-5)
    ga = torch.ones(H, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    want = xh * ga + (0 if beta is None else beta.double())
    _close(y, want, e * ga.abs() + U * ((xh * ga).abs() + want.abs()))
    _close(mean, m[:, 0], 46 * U / q[:, 0])
    _close(rstd, q[:, 0], 30 * U * q[:, 0])
    if pad:
        assert torch.isnan(out.as_strided((T, pad), (H + pad, 1), out.storage_offset() + H)).all()
    made, none, none2 = op(x, stats=False)
    assert torch.equal(made, out) and none is None and none2 is None
    if xt is yt and not pad:                               # in place
        x2 = x.clone()
        op(x2, out=x2)
        assert torch.equal(x2, out)


@pytest.mark.parametrize("case", _CASES, ids=_ID)
def test_layer_norm_backward(case):
    T, H, xt, yt, _, _, pad, _ = case
    gen, x, gamma, beta, op = _make(case)
    dy, add = _rows(T, H, pad, yt, gen), _rows(T, H, pad, xt, gen)
    m, q, xh, e = _stats(x, 1e-5)
    mean, rstd = m[:, 0].float(), q[:, 0].float()
    dg, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    dx, dg2, db2 = op.backward(dy, x, mean, rstd, add=add, dx=_rows(T, H, pad, xt, gen), dgamma=dg, dbeta=db)
    assert dg2 is dg and db2 is db
    d = dy.double()
    ga = torch.ones(H, device="cuda", dtype=torch.float64) if gamma is None else gamma.double()
    g = d * ga
    mg, mgx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx0 = q * (g - mg - xh * mgx)
    ag, agx, age = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True), (g.abs() * e).mean(1, keepdim=True)
    tol = q * (44 * U * (ag + xh.abs() * agx) + xh.abs() * age + e * mgx.abs() + 4 * U * (g.abs() + mg.abs() + (xh * mgx).abs()))
    want = dx0 + add.double()
    _close(dx, want, tol + U * (add.double().abs() + want.abs()))
    depth = U * (T / 150 + 66)
    _close(dg, (d * xh).sum(0), depth * (d * xh).abs().sum(0) + (d.abs() * e).sum(0))
    _close(db, d.sum(0), depth * d.abs().sum(0))
    if pad:
        assert torch.isnan(dx.as_strided((T, pad), (H + pad, 1), dx.storage_offset() + H)).all()
    # without the residual stream's gradient; into dy's or add's own memory; sums added to what is there; alone
    plain, _, _ = op.backward(dy, x, mean, rstd)
    _close(plain, dx0, tol + U * dx0.abs())
    a2 = add.clone() if not pad else add
    keep = dx.clone()
    op.backward(dy, x, mean, rstd, add=a2, dx=a2, dgamma=dg, dbeta=db, accumulate=True)
    assert torch.equal(a2, keep)
    _close(dg, 2 * (d * xh).sum(0), 2 * depth * (d * xh).abs().sum(0) + 2 * (d.abs() * e).sum(0) + 2 * U * dg.double().abs())
    _close(db, 2 * d.sum(0), 2 * depth * d.abs().sum(0) + 2 * U * db.double().abs())


@pytest.mark.parametrize("H", [96, 2048, 9000])
def test_layer_norm_gradient_against_differences(H):
    """Central differences of the forward formula in 64 bits, along random directions of x, gamma and beta: with steps of
    h = 1e-4 they are off by h^2 / 6 times a third derivative of order 1 (1e-8 here); the kernel's fp32 sums by 1e-5."""
    T = 6
    gen = torch.Generator(device="cuda").manual_seed(H)
    x = _rows(T, H, 0, F32, gen)
    gamma, beta = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda"), torch.randn(H, generator=gen, device="cuda")
    w = _rows(T, H, 0, F32, gen)
    op = moe.LayerNorm(H, gamma=gamma, beta=beta, y_dtype=F32)
    _, mean, rstd = op(x)
    dx, dg, db = op.backward(w, x, mean, rstd)

    def loss(x, ga, be):
        m = x.mean(1, keepdim=True)
        return ((x - m) / ((x - m).pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * ga + be).mul(w.double()).sum()

    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate((dx, dg, db)):
        v = torch.randn(args[i].shape, generator=gen, device="cuda").double()
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - 1e-4 * v, args[i] + 1e-4 * v
        diff = (loss(*hi) - loss(*lo)) / 2e-4
        assert abs(diff - (grad.double() * v).sum()) <= 1e-5 * (grad.double() * v).norm() + 1e-6 * w.double().norm()


def test_layer_norm_zero_rows_infinities_and_nan():
    H = 96
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = _rows(5, H, 0, F32, gen)
    x[2] = 3.5                                              # a constant row: xh = 0, rstd = 1 / sqrt(eps)
    beta = torch.randn(H, generator=gen, device="cuda")
    op = moe.LayerNorm(H, beta=beta, y_dtype=F32)
    y, mean, rstd = op(x)
    assert torch.equal(y[2], beta) and mean[2] == 3.5 and abs(rstd[2].item() * 1e-5 ** 0.5 - 1) < 1e-6
    x2 = x.clone()
    x2[1, 5], x2[3, 0] = float("nan"), float("inf")
    y2, mean2, rstd2 = op(x2)
    keep = [0, 2, 4]
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[1]).all() and torch.isnan(y2[3]).all()
    assert torch.isnan(rstd2[[1, 3]]).all() and torch.isnan(mean2[1])


def test_layer_norm_without_rows():
    H = 64
    op = moe.LayerNorm(H, gamma=torch.ones(H, device="cuda"), beta=torch.ones(H, device="cuda"))
    x = torch.zeros(0, H, device="cuda")
    y, mean, rstd = op(x)
    assert y.shape == (0, H) and mean.shape == (0,)
    dg, db = torch.full((H,), 7.0, device="cuda"), torch.full((H,), 7.0, device="cuda")
    op.backward(y, x, mean, rstd, dgamma=dg, dbeta=db, accumulate=True)
    assert bool((dg == 7).all()) and bool((db == 7).all())
    op.backward(y, x, mean, rstd, dgamma=dg, dbeta=db)
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_layer_norm_captured_two_at_once_and_on_another_stream():
    T, H = 700, 1024
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, dy = _rows(T, H, 0, F32, gen), _rows(T, H, 0, BF, gen)
    gamma = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda")
    op = moe.LayerNorm(H, gamma=gamma, beta=gamma)

    def step(s=None):
        y, mean, rstd = op(x, stream=s)
        return (y, mean, rstd) + op.backward(dy, x, mean, rstd, stream=s)

    ref = [t.clone() for t in step()]
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            outs.append(step())
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = step(streams[2])
        torch.cuda.synchronize()
        for got in outs + [eager]:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_layer_norm_of_rows_that_lie_far_apart():
    """Strides of 2^31 + 8 elements: offsets beyond 32 bits in elements and bytes."""
    T, H, far = 3, 264, (1 << 31) + 8
    gen = torch.Generator(device="cuda").manual_seed(4)
    gamma = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda")
    op = moe.LayerNorm(H, gamma=gamma, beta=gamma)
    x0, d0 = (torch.randn(T, H, generator=gen, device="cuda").to(BF) for _ in range(2))
    want, mean, rstd = op(x0)
    sums = op.backward(d0, x0, mean, rstd, add=d0)
    buf = torch.empty(2 * far + 4 * H, dtype=BF, device="cuda")
    x, y, dy, dx = (buf[i * H:].as_strided((T, H), (far, 1)) for i in range(4))
    x.copy_(x0)
    dy.copy_(d0)
    op(x, out=y)
    got = op.backward(dy, x, mean, rstd, add=dy, dx=dx)
    assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(got, sums))
