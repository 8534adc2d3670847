"""The norms around a block (moe_norm_residual) on the GPU against the formula in 64 bits.

Tolerance, before any run.  A mean of H squares in fp32: a thread adds at most 32 of them one after another, the
rest is a tree of at most 12 levels, so the sum of positive terms is off by at most 44 * 2^-24 relative; its
inverse root halves that and adds 3 roundings: e = 26 * 2^-24.  n then has 3 more roundings, the gate and the
scales 3: |r error| <= (e + 6 * 2^-24) |scale gate n| + 2^-24 (|res_scale x| + |r|) <= 34 * 2^-24 (|scale gate n| + |res_scale x|) =: d.
u = r f with f = gamma / rms: |u error| <= d f + |u| (e + 3 * 2^-24 + D), D the relative error of the root mean of
r, at most the root mean square of d over that of r.  Storing adds half a step of the output's type.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _rows(T, H, pad, dtype, gen, scale):
    full = torch.full((T, H + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :H] = torch.randn(T, H, generator=gen, device="cuda") * scale
    return full[:, :H]


def _want(x, y, gp, gate, ga, eps, rs, sc):
    v = y.double()
    if gp is not None:
        v = v / (v.pow(2).mean(1, keepdim=True) + eps).sqrt() * gp.double()
    if gate is not None:
        v = v * gate.double()
    v = sc * v
    xr = torch.zeros_like(v) if x is None else rs * x.double()
    r = v + xr
    d = 34 * 2.0 ** -24 * (v.abs() + xr.abs())
    if ga is None:
        return r, d, None, None
    root = (r.pow(2).mean(1, keepdim=True) + eps).sqrt()
    f = ga.double() / root
    u = r * f
    D = d.pow(2).mean(1, keepdim=True).sqrt() / root
    return r, d, u, d * f.abs() + u.abs() * (29 * 2.0 ** -24 + D)


def _close(got, want, tol):
    t = got.dtype
    tol = tol + torch.finfo(t).eps / 2 * (want.abs() + tol) + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() - tol).max()


_CASES = [
    # T, H, x type, y type, u type, post, gate, pad
    (1, 1, F32, F32, BF, True, None, 0),
    (1, 2048, F32, F32, BF, True, None, 0),
    (3, 7, BF, F32, HF, True, "channel", 0),
    (5, 64, F32, BF, BF, False, "token", 0),
    (19, 256, HF, HF, HF, True, "full", 8),
    (70, 264, BF, BF, BF, True, "channel", 8),
    (9, 512, F32, F32, F32, True, "full", 0),
    (7, 768, BF, F32, BF, True, "channel", 0),
    (4, 1024, F32, BF, BF, True, None, 8),
    (5, 1023, F32, F32, BF, True, "token", 0),
    (33, 1000, F32, BF, BF, True, "token", 3),
    (4, 2047, BF, BF, BF, True, "full", 1),
    (300, 2048, F32, F32, BF, True, None, 0),
    (6, 4096, F32, F32, BF, True, "channel", 0),
    (6, 4095, HF, F32, F32, False, None, 0),
    (40, 7168, BF, BF, BF, True, "channel", 8),
    (3, 7169, F32, BF, HF, True, "full", 0),
    (2, 16384, F32, F32, BF, True, None, 0),
    (2, 16383, BF, BF, BF, True, "token", 0),
    (2, 32768, F32, F32, BF, True, "channel", 0),
    (2, 32767, F32, F32, F32, True, "full", 0),
]


@pytest.mark.parametrize("case", _CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_norm_residual(case):
    T, H, xt, yt, ut, post, gk, pad = case
    gen = torch.Generator(device="cuda").manual_seed(H * 7 + T)
    x, y = _rows(T, H, pad, xt, gen, 2.0), _rows(T, H, pad, yt, gen, 0.3)
    gp = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")) if post else None
    ga = 1 + 0.1 * torch.randn(H, generator=gen, device="cuda")
    shape = {None: None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gk]
    gate = torch.rand(shape, generator=gen, device="cuda") if shape else None
    op = moe.NormResidual(H, gamma_post=gp, gamma_pre=ga, eps=1e-5, res_scale=0.75, scale=1.5)
    xo, u = _rows(T, H, pad, xt, gen, 1.0), _rows(T, H, pad, ut, gen, 1.0)
    a, b = op(x, y, gate, x_out=xo, u=u)
    assert a is xo and b is u
    torch.cuda.synchronize()
    r, d, w, dw = _want(x, y, gp, gate, ga, 1e-5, 0.75, 1.5)
    _close(xo, r, d)
    _close(u, w, dw)
    if pad:                                                # what lies between the rows is left alone
        for t in (xo, u):
            assert torch.isnan(t.as_strided((T, pad), (H + pad, 1), t.storage_offset() + H)).all()
    before_x, before_u = xo.clone(), u.clone()             # in place, and each output alone: the same bits
    x2 = x.clone()
    op(x2, y, gate, x_out=x2, u=u)
    assert torch.equal(x2, before_x) and torch.equal(u, before_u)
    only = moe.NormResidual(H, gamma_post=gp, eps=1e-5, res_scale=0.75, scale=1.5)
    got, none = only(x, y, gate)
    assert none is None and torch.equal(got, before_x)


def test_norm_without_a_residual_and_of_zeros():
    H = 96
    gen = torch.Generator(device="cuda").manual_seed(2)
    y = _rows(4, H, 0, F32, gen, 1.0)
    y[2] = 0.0                                              # a row of zeros: 0 / sqrt(eps) = 0
    ga = torch.ones(H, device="cuda")
    op = moe.NormResidual(H, gamma_post=ga, gamma_pre=ga, eps=1e-6)
    r, u = op(None, y)
    want, d, w, dw = _want(None, y, ga, None, ga, 1e-6, 1.0, 1.0)
    _close(r, want, d)
    _close(u, w, dw)
    assert bool((r[2] == 0).all()) and bool((u[2] == 0).all())
    y[1, 5] = float("nan")
    y[3, 0] = float("inf")
    r2, u2 = op(None, y)
    assert torch.equal(r2[[0, 2]], r[[0, 2]]) and torch.equal(u2[[0, 2]], u[[0, 2]])
    assert bool(torch.isnan(u2[1]).all()) and bool(torch.isnan(r2[3, 0]))


def test_norm_matches_the_layer_norm():
    """With no block norm, no gate and unit scales u is what moe_rmsnorm_bf16 gives for x + y (same definition)."""
    T, H = 5, 2048
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, y = _rows(T, H, 0, F32, gen, 1.0), _rows(T, H, 0, F32, gen, 1.0)
    ga = 1 + 0.01 * torch.randn(H, generator=gen, device="cuda")
    r, u = moe.NormResidual(H, gamma_pre=ga, eps=1e-6)(x, y)
    assert torch.equal(r, x + y)
    v = torch.empty(T, H, dtype=BF, device="cuda")
    moe.moe_rmsnorm_bf16(r, ga, T, H, 1e-6, v)
    # the two sum the squares in different orders: at most one bf16 step apart, on few elements
    diff = (u.float() - v.float()).abs()
    assert bool((diff <= 2.0 ** -7 * v.float().abs()).all()) and (diff > 0).float().mean() < 0.01


def test_norm_captured_and_replayed():
    T, H = 7, 1024
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, y = _rows(T, H, 0, F32, gen, 1.0), _rows(T, H, 0, BF, gen, 1.0)
    ga = torch.ones(H, device="cuda")
    op = moe.NormResidual(H, gamma_post=ga, gamma_pre=ga)
    xo, u = torch.empty_like(x), torch.empty(T, H, dtype=BF, device="cuda")
    op(x, y, x_out=xo, u=u)
    ref = xo.clone(), u.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        op(x, y, x_out=xo, u=u)
    xo.zero_()
    u.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(xo, ref[0]) and torch.equal(u, ref[1])
