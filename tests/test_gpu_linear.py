"""The dense product with its epilogue (moe_linear) on the GPU against the formula in 64 bits.

Tolerance, per element and before any run.  Products of two 16-bit numbers are exact in fp32.  A term passes through
at most `depth` additions: the matrix instructions that follow one another in its run (one per 16 terms, a run of at
most 768 terms for fp32 outputs and 8192 for 16-bit ones), the terms inside one instruction, the runs and the 8 parts of a
split sum.  Each is off by at most 2^-23 of the largest partial sum, which is at most A = sum |w x|:
|z error| <= depth 2^-23 A + 2^-24 |z| (the bias).  No activation is steeper than 1.13; its own error is at most 2e-5 of
its value for 16-bit outputs (a 20th of half a step of fp16) and 16 * 2^-24 for fp32 ones (exponential, normal
distribution function, division: a few units each), of the slope's value where z is near 0.  Scale, residual
and sum add a rounding each.  Storing adds half a step of the output's type.
"""
from __future__ import annotations

import math

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0.0), "silu": lambda v: v * torch.sigmoid(v),
        "gelu": lambda v: v * 0.5 * torch.erfc(v * -math.sqrt(0.5)),
        "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(gen, n, width, stride, dtype, scale=1.0):
    full = torch.full((n, stride), float("nan"), dtype=dtype, device="cuda")
    full[:, :width] = torch.randn(n, width, generator=gen, device="cuda") * scale
    return full[:, :width]


def _pad8(n):
    return -(-n // 8) * 8


def _want(x, w, order, bias, act, scale, r, res_scale, y_dtype):
    m = w.double() if order == "out_in" else w.double().t()
    z, A = x.double() @ m.t(), x.double().abs() @ m.double().abs().t()
    K = x.shape[1]
    depth = min(-(-K // 16), 48 if y_dtype is F32 else 512) + 16 + -(-K // 768) + 8
    if bias is not None:
        z, A = z + bias.double(), A + bias.double().abs()
    dz = depth * 2.0 ** -23 * A + 2.0 ** -24 * z.abs()
    a = ACTS[act](z)
    da = 1.13 * dz + (0.0 if act in ("none", "relu") else 16 * 2.0 ** -24 if y_dtype is F32 else 2e-5) * a.abs()
    want, tol = scale * a, abs(scale) * da + 2.0 ** -24 * abs(scale) * a.abs()
    if r is not None:
        want = want + res_scale * r.double()
        tol = tol + 2.0 ** -23 * (res_scale * r.double()).abs() + 2.0 ** -24 * want.abs()
    return want, tol


def _close(got, want, tol):
    t = got.dtype
    tol = tol + torch.finfo(t).eps / 2 * (want.abs() + tol) + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    bad = (got.double() - want).abs() - tol
    assert not torch.isnan(got).any() and (bad <= 0).all(), (bad.max(), int((bad > 0).sum()))


def _check(T, K, N_, x_dtype, y_dtype, act, bias, res, order, pad, path=None, seed=0):
    gen = _gen(T + 3 * K + 7 * N_ + seed)
    x = _rows(gen, T, K, _pad8(K) + 8 * pad, x_dtype)
    a, b = (N_, K) if order == "out_in" else (K, N_)
    w = _rows(gen, a, b, _pad8(b) + 8 * pad, x_dtype, 1 / math.sqrt(K))
    bt = torch.randn(N_, generator=gen, device="cuda").to(bias) if bias else None
    r = _rows(gen, T, N_, N_ + pad, res, 2.0) if res else None
    op = moe.Linear(w, bt, order=order, act=act, y_dtype=y_dtype, scale=1.25, res_scale=0.5)
    assert path is None or op.path(T) == path
    out = _rows(gen, T, N_, N_ + pad, y_dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert op(x, residual=r, out=out, status=status) is out
    torch.cuda.synchronize()
    assert status.item() == N.MOE_OK
    _close(out, *_want(x, w, order, bt, act, 1.25, r, 0.5, y_dtype))
    if pad:                                                # what lies between the rows is left alone
        assert torch.isnan(out.as_strided((T, pad), (N_ + pad, 1), out.storage_offset() + N_)).all()
    assert torch.equal(op(x, residual=r), out)
    if res is y_dtype:                                     # in place: the same bits
        r2 = r.as_strided((T, N_), r.stride()).clone() if not pad else _rows(gen, T, N_, N_ + pad, res).copy_(r)
        op(x, residual=r2, out=r2)
        assert torch.equal(r2, out)


@pytest.mark.parametrize("order", ["out_in", "in_out"])
@pytest.mark.parametrize("T, K, N_", [(1, 1, 1), (1, 64, 128), (1, 2048, 2048), (2, 7, 5), (1, 768, 40), (3, 776, 129), (16, 100, 333),
                                      (17, 1000, 127), (31, 4099, 256), (33, 65, 1000), (64, 2048, 768), (65, 130, 257),
                                      (128, 512, 384), (129, 513, 641), (500, 5000, 100), (600, 96, 72)])
@pytest.mark.parametrize("y", [F32, BF])
def test_linear_sizes(order, T, K, N_, y):
    _check(T, K, N_, BF, y, "gelu", F32, y, order, 0, "split")
    _check(T, K, N_, HF if y is BF else BF, y if y is F32 else HF, "none", None, None, order, 3, "split")


@pytest.mark.parametrize("order", ["out_in", "in_out"])
@pytest.mark.parametrize("T, K, N_", [(300, 1000, 1333), (1000, 100, 3100), (1537, 2048, 2048), (4097, 72, 700), (256, 776, 12300), (12400, 65, 130),
                                      (2000, 9000, 1600)])
@pytest.mark.parametrize("y", [F32, BF])
def test_linear_pairs(order, T, K, N_, y):
    _check(T, K, N_, BF, y, "silu", BF, F32, order, 1, "pairs")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("x, y", [(BF, BF), (HF, HF), (BF, F32), (HF, BF)])
@pytest.mark.parametrize("T", [5, 2100])
def test_linear_activations_and_types(act, x, y, T):
    for bias, res in ((F32, HF), (BF, BF), (HF, F32), (None, None)):
        _check(T, 200, 1500, x, y, act, bias, res, "out_in", 0)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("y", [F32, HF, BF])
def test_linear_activation_over_its_range(act, y):
    """z from -120 to 120 through the bias: the tails of the activations, where they are far below z."""
    N_ = 4801
    w = torch.zeros(N_, 8, dtype=BF, device="cuda")
    bias = torch.linspace(-120, 120, N_, device="cuda")
    x = torch.ones(3, 8, dtype=BF, device="cuda")
    got = moe.Linear(w, bias, act=act, y_dtype=y)(x)
    z = bias.double()
    want = ACTS[act](z)
    # (fp32: normcdf's and the exponential's own errors grow with z^2; their results below 2^-126 have that spacing)
    # (the exponential of -w, w = z^2 / 2, 1.6 (z + 0.044715 z^3) or z: relative error at most (2 + 1.2 w + w) 2^-23, w <= 90 where
    # the result is not 0: 2.4e-5)
    tol = 2.6e-5 * want.abs() + 2.0 ** -126 * z.abs()
    half = torch.finfo(y).eps / 2
    step = torch.finfo(y).smallest_normal * torch.finfo(y).eps
    assert ((got.double() - want).abs() <= tol + half * want.abs() * 1.001 + step).all()


def test_linear_infinities_and_nan_stay_in_their_row_and_channel():
    gen = _gen(1)
    x = torch.randn(40, 200, generator=gen, device="cuda").to(BF)
    w = torch.randn(300, 200, generator=gen, device="cuda").to(BF)
    r = torch.randn(40, 300, generator=gen, device="cuda")
    op = moe.Linear(w, None, act="relu", y_dtype=F32)
    ref = op(x, residual=r)
    x2, r2, w2 = x.clone(), r.clone(), w.clone()
    x2[7, 3] = float("nan")
    r2[9, 11] = float("inf")
    got = op(x2, residual=r2)
    rows = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(got[rows], ref[rows]) and torch.isnan(got[7]).all() and got[9, 11] == float("inf")
    w2[123, 5] = float("nan")
    got = moe.Linear(w2, None, act="relu", y_dtype=F32)(x, residual=r)
    assert torch.isnan(got[:, 123]).all() and torch.equal(got[:, :123], ref[:, :123]) and torch.equal(got[:, 124:], ref[:, 124:])


@pytest.mark.parametrize("T, N_", [(4, 200), (300, 200), (2000, 1600)])
@pytest.mark.parametrize("K", [768, 2048, 7168, 65536])
def test_linear_long_sums_keep_their_precision(T, N_, K):
    """fp32 outputs: the error does not grow with the number of matrix instructions.

    Relative in norm, before any run: a run of 48 instructions that cut off is off by at most 48 * 2^-24 * 2/3 of its sum, and so
    is a sum of runs; up to 86 runs and 8 parts added with rounding and the terms inside an instruction: 64 * 2^-24 / 4.
    """
    if T * K > 1 << 24:
        T = 300
    gen = _gen(K)
    x = torch.randn(T, K, generator=gen, device="cuda").abs().to(BF)
    w = torch.randn(N_, K, generator=gen, device="cuda").abs().to(BF)
    got = moe.Linear(w, y_dtype=F32)(x).double()
    want = x.double() @ w.double().t()
    assert ((got - want).norm() / want.norm()).item() <= (48 * 2 / 3 + 16) * 2.0 ** -24


@pytest.mark.parametrize("T, N_", [(1, 300), (40, 2048), (2000, 1600)])
def test_linear_captured_two_at_once_and_on_another_stream(T, N_):
    gen = _gen(4)
    K = 1024
    a, b = (moe.Linear(torch.randn(N_, K, generator=gen, device="cuda").to(BF), act="gelu") for _ in range(2))
    x = torch.randn(T, K, generator=gen, device="cuda").to(BF)
    ra, rb = a(x), b(x)
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga, stream=torch.cuda.Stream()):
        a(x, out=oa)
    with torch.cuda.graph(gb, stream=torch.cuda.Stream()):
        b(x, out=ob)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        oa.zero_(), ob.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            ga.replay()
            c = b(x, stream=s)
        with torch.cuda.stream(t):
            gb.replay()
            d = a(x, stream=t.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb) and torch.equal(c, rb) and torch.equal(d, ra)
    assert a.device_status() == b.device_status() == N.MOE_OK


def test_linear_columns_of_one_buffer():
    T, K, N_ = 200, 64, 72
    gen = _gen(6)
    op = moe.Linear(torch.randn(N_, K, generator=gen, device="cuda").to(BF), act="silu")
    values, res = torch.randn(T, K, generator=gen, device="cuda").to(BF), torch.randn(T, N_, generator=gen, device="cuda").to(BF)
    want = op(values, residual=res)
    buf = torch.full((T, K + 2 * N_ + 8), 7.0, dtype=BF, device="cuda")
    x, y, r = buf[:, :K], buf[:, K: K + N_], buf[:, K + N_: K + 2 * N_]
    x.copy_(values)
    r.copy_(res)
    op(x, residual=r, out=y)
    assert torch.equal(y, want) and torch.equal(x, values) and torch.equal(r, res) and bool((buf[:, K + 2 * N_:] == 7.0).all())


@pytest.mark.parametrize("T, N_, path", [(3, 300, "split"), (3, 5000, "split"), (200, 2048, "split"), (2000, 1600, "pairs")])
def test_linear_wait_that_runs_out_is_reported(T, N_, path):
    gen = _gen(9)
    K = 4096
    op = moe.Linear(torch.randn(N_, K, generator=gen, device="cuda").to(BF), y_dtype=F32)
    assert op.path(T) == path
    x = torch.randn(T, K, generator=gen, device="cuda").to(BF)
    ref = op(x).clone()
    torch.cuda.synchronize()
    try:
        N.moe_debug_set_waits(2_000_000, 1)
        op(x)
        torch.cuda.synchronize()
    finally:
        N.moe_debug_set_waits(0, 0)
    assert op.device_status(clear=True) == N.MOE_ERR_TIMEOUT
    assert torch.equal(op(x), ref) and op.device_status() == N.MOE_OK


def test_linear_without_rows():
    op = moe.Linear(torch.zeros(16, 32, dtype=BF, device="cuda"))
    assert op(torch.zeros(0, 32, dtype=BF, device="cuda")).shape == (0, 16)


@pytest.mark.parametrize("T, N_", [(3, 200), (2000, 1600)])
def test_linear_of_rows_that_lie_far_apart(T, N_):
    """Offsets beyond 32 bits: x, residual and y of one buffer, its rows 2^31 + 8 elements (3 rows) or 2^22 + 8 elements apart."""
    K, far = 96, (1 << 31) + 8 if T == 3 else (1 << 22) + 8
    gen = _gen(2)
    op = moe.Linear(torch.randn(N_, K, generator=gen, device="cuda").to(BF), act="silu")
    x0, r0 = torch.randn(T, K, generator=gen, device="cuda").to(BF), torch.randn(T, N_, generator=gen, device="cuda").to(BF)
    want = op(x0, residual=r0)
    buf = torch.empty((T - 1) * far + K + 2 * N_, dtype=BF, device="cuda")
    x, r, y = (buf[i:].as_strided((T, w), (far, 1)) for i, w in ((0, K), (K, N_), (K + N_, N_)))
    x.copy_(x0)
    r.copy_(r0)
    op(x, residual=r, out=y)
    assert torch.equal(y, want)
