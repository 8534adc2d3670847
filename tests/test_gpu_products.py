"""Grouped products (bf16 / fp16 weights) and 4-bit products on the GPU against the formula in 64 bits.

Tolerance, per element and before any run.  Products of two 16-bit numbers (or of a 16-bit number
and a code of at most 5 bits) are exact in fp32.  A term passes through at most `depth` additions: the
matrix instructions that follow one another in its sum (one per 16 terms; the rows kernel shares them among 8
warps, the tensor kernel does not), the terms inside one instruction, and the join.  Each addition is
off by at most 2^-23 of the largest partial sum (a truncating adder loses one unit, a rounding one half), which
is at most A = sum |w x|: |error| <= depth * 2^-23 * A.  The scale of a 4-bit group is one more rounding (in
the depth).  Storing adds half a step of the output's type.  For the gated pair the error of g passes through silu
(slope at most 1.1) times u, that of u through silu(g); exp, the division and the product add a few
roundings of the result (8 * 2^-24).
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _routing(sizes, T, k, gen):
    """offsets of the given sizes and pairs p (every expert's ascending) so that row i reads token p // k."""
    P = T * k
    assert sum(sizes) <= P
    off = torch.zeros(len(sizes) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(sizes, dtype=torch.int32), 0)
    pairs = torch.randperm(P, generator=torch.Generator().manual_seed(T * 31 + k)).to(torch.int32)
    return off.cuda(), pairs.cuda()


def _split(P, E, seed):
    """Sizes of E experts with P rows in all: some empty, uneven."""
    g = torch.Generator().manual_seed(seed)
    p = 1.0 / torch.arange(1, E + 1) ** 1.2
    p = p[torch.randperm(E, generator=g)]
    if E > 2:
        p[torch.randperm(E, generator=g)[: E // 3]] = 0.0
    ids = torch.multinomial(p, P, replacement=True, generator=g)
    return torch.bincount(ids, minlength=E).tolist()


def _finish(g, ga, u, ua, depth):
    """(expected, tolerance) of the sums g, u with absolute sums ga, ua."""
    step = depth * 2.0 ** -23
    if u is None:
        return g, step * ga
    s = g / (1 + torch.exp(-g))
    want = s * u
    return want, 1.1 * step * ga * u.abs() + s.abs() * step * ua + step * ga * step * ua * 1.1 + 8 * 2.0 ** -24 * want.abs()


def _expected(x, w, w_up, off, rows):
    """Row by row: the sums and absolute sums in 64 bits.  w: function (expert) -> [N, K] double."""
    out = [[], [], [], []]
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        v = x.double()[rows[a:b]]
        m = w(e)
        out[0].append(v @ m.t())
        out[1].append(v.abs() @ m.abs().t())
        if w_up is not None:
            m = w_up(e)
            out[2].append(v @ m.t())
            out[3].append(v.abs() @ m.abs().t())
    return [torch.cat(o) if o else None for o in out]


def _close(got, want, tol, dtype, what=""):
    tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(got).any(), what
    assert off.max().item() <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()} beyond the tolerance by up to {off.max():.3g}"


def _rows_of(gather, off, pairs, k):
    P = off[-1]
    return (pairs.long() // k) if gather else torch.arange(max(P, 1), device="cuda")


def _padded(n, width, pad, dtype, gen, scale=1.0, fill=None):
    stride = -(-width // 8) * 8 + pad
    full = torch.empty(n, stride, dtype=dtype, device="cuda").normal_(0, scale, generator=gen)
    if fill is not None:
        full[:, width:] = fill
    return full[:, :width]


def _dense_case(T, k, E, K, N_, up, gather, dtype, y_dtype, order, pad=0, sizes=None, seed=0):
    gen = _gen(seed + 17)
    sizes = _split(T * k, E, seed) if sizes is None else sizes
    off, pairs = _routing(sizes, T, k, gen)
    # what lies between the rows must not matter: NaN there
    x = _padded(T if gather else T * k, K, pad, dtype, gen, fill=float("nan"))
    a, b = (N_, K) if order == "out_in" else (K, N_)
    make = lambda: _padded(E * a, b, pad, dtype, gen, 0.05, float("nan")).unflatten(0, (E, a))  # noqa: E731
    w, w_up = make(), (make() if up else None)
    return sizes, off, pairs, x, w, w_up


def _run_dense(op, T, k, N_, up, gather, off, pairs, x, w, w_up, order, y_dtype, y_pad=0, depth=None):
    P = T * k
    full = torch.full((P, N_ + y_pad), 7.0, dtype=y_dtype, device="cuda")
    y = full[:, :N_]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    op(x, off, pairs if gather else None, k=k, out=y, status=status)
    torch.cuda.synchronize()
    assert status.item() == N.MOE_OK
    o = off.tolist()
    get = lambda m: (lambda e: m[e].double() if order == "out_in" else m[e].double().t())  # noqa: E731
    K = x.shape[1]
    g, ga, u, ua = _expected(x, get(w), get(w_up) if up else None, o, _rows_of(gather, o, pairs, k))
    # nothing outside the experts' rows and columns is written
    assert bool((full[:, N_:] == 7.0).all())
    assert bool((full[o[-1]:] == 7.0).all())
    if o[-1] == 0:
        return y
    depth = K // 16 + 40 if depth is None else depth
    want, tol = _finish(g, ga, u, ua, depth)
    _close(y[: o[-1]], want, tol, y_dtype)
    return y


_DENSE = [
    # T, k, E, K, N, up, gather, x dtype, y dtype, order, pad
    (1, 1, 1, 1, 1, False, False, BF, F32, "out_in", 0),
    (1, 1, 1, 7, 5, True, False, HF, F32, "out_in", 8),
    (1, 2, 4, 64, 32, False, True, BF, BF, "out_in", 0),
    (1, 8, 128, 256, 96, True, True, BF, BF, "out_in", 0),
    (3, 2, 5, 100, 33, True, True, BF, F32, "out_in", 8),
    (9, 2, 3, 333, 65, False, True, HF, HF, "out_in", 16),
    (17, 1, 2, 128, 64, True, False, HF, F32, "out_in", 0),
    (40, 4, 6, 200, 130, True, True, BF, BF, "out_in", 8),
    (64, 8, 16, 512, 48, False, False, BF, F32, "out_in", 0),
    (130, 3, 7, 1000, 77, True, True, HF, HF, "out_in", 24),
    (300, 4, 5, 64, 256, False, True, BF, F32, "out_in", 0),
    (700, 2, 3, 96, 300, True, True, BF, BF, "out_in", 0),
    (5, 2, 1024, 32, 16, False, True, BF, F32, "out_in", 0),
    (600, 3, 1024, 40, 24, False, True, BF, F32, "out_in", 0),
    (1, 1, 1, 1, 1, False, False, HF, F32, "in_out", 0),
    (1, 8, 16, 256, 96, True, True, BF, BF, "in_out", 0),
    (3, 2, 5, 100, 33, True, True, BF, F32, "in_out", 8),
    (20, 2, 3, 77, 130, False, True, HF, HF, "in_out", 16),
    (40, 4, 6, 200, 130, True, False, BF, BF, "in_out", 8),
    (300, 4, 5, 64, 256, False, True, BF, F32, "in_out", 0),
    (700, 2, 3, 96, 300, True, True, HF, HF, "in_out", 0),
    (2048, 1, 1, 128, 128, False, False, BF, F32, "out_in", 0),
]


@pytest.mark.parametrize("case", _DENSE, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_grouped_products(case):
    T, k, E, K, N_, up, gather, dtype, y_dtype, order, pad = case
    sizes, off, pairs, x, w, w_up = _dense_case(*case, seed=len(str(case)))
    op = moe.GroupedExperts(w, w_up, order=order, y_dtype=y_dtype)
    _run_dense(op, T, k, N_, up, gather, off, pairs, x, w, w_up, order, y_dtype, y_pad=pad // 8)


@pytest.mark.parametrize("sizes", [[0, 0, 0], [12, 0, 0], [0, 0, 12], [0, 12, 0], [1, 1, 1], [4, 0, 5], [0, 1, 0]])
@pytest.mark.parametrize("up", [False, True])
def test_grouped_rows_that_end_early(sizes, up):
    """Empty experts, and rows of y behind the last expert (as moe_permute leaves them for dropped pairs)."""
    T, k, E, K, N_ = 6, 2, 3, 72, 40
    _, off, pairs, x, w, w_up = _dense_case(T, k, E, K, N_, up, True, BF, F32, "out_in", 0, sizes)
    op = moe.GroupedExperts(w, w_up, y_dtype=F32)
    _run_dense(op, T, k, N_, up, True, off, pairs, x, w, w_up, "out_in", F32)


def test_grouped_one_expert_without_offsets():
    for T, K, N_ in ((1, 96, 50), (45, 96, 50), (400, 96, 50)):
        _, _, _, x, w, _ = _dense_case(T, 1, 1, K, N_, False, False, BF, F32, "out_in")
        op = moe.GroupedExperts(w)
        off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        a, b = op(x), op(x, off)
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [2, 300])
def test_grouped_bad_routing_is_reported(T):
    """Offsets and pairs outside their range are clamped and reported; nothing is read or written out of range."""
    k, E, K, N_ = 2, 3, 64, 32
    _, off, pairs, x, w, _ = _dense_case(T, k, E, K, N_, False, True, BF, F32, "out_in", sizes=[T, T, 0])
    op = moe.GroupedExperts(w)
    good = op(x, off, pairs, k=k).clone()
    for which in ("offset above", "offset below", "pair above", "pair below"):
        o, p = off.clone(), pairs.clone()
        if which == "offset above":
            o[3] = 2 * T + 5
            o[2] = 2 * T
        elif which == "offset below":
            o[0] = -3
        else:
            p[1] = 2 * T if which == "pair above" else -1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = op(x, o, p, k=k, status=status)
        torch.cuda.synchronize()
        assert status.item() == N.MOE_ERR_DEVICE_CHECK, which
        keep = torch.ones(2 * T, dtype=torch.bool, device="cuda")
        if which.startswith("pair"):
            keep[1] = False
        assert torch.equal(y[keep], good[keep]), which
        op(x, off, pairs, k=k, status=status)              # not cleared by the next good call
        torch.cuda.synchronize()
        assert status.item() == N.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("T", [4, 200])
@pytest.mark.parametrize("order", ["out_in", "in_out"])
def test_grouped_nan_and_inf_stay_in_their_row(T, order):
    """A row of x that is not finite spoils its own row of y only; a weight that is not, its own column."""
    _, off, pairs, x, w, _ = _dense_case(T, 1, 2, 80, 48, False, False, BF, F32, order, sizes=[T // 2, T - T // 2])
    op = moe.GroupedExperts(w, order=order)
    good = op(x, off).clone()
    x[1, 3], x[T - 1, 79] = float("nan"), float("inf")
    bad = op(x, off)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1] = keep[T - 1] = False
    assert torch.equal(bad[keep], good[keep])
    assert bool(torch.isnan(bad[1]).all()) and not bool(torch.isfinite(bad[T - 1]).any())
    x[1, 3], x[T - 1, 79] = 0.0, 0.0
    base = op(x, off).clone()
    if order == "out_in":
        w[0, 5, 70] = float("nan")
    else:
        w[0, 70, 5] = float("nan")
    bad = op(x, off)
    assert bool(torch.isnan(bad[: T // 2, 5]).all())
    cols = [c for c in range(48) if c != 5]
    assert torch.equal(bad[:, cols], base[:, cols]) and torch.equal(bad[T // 2:], base[T // 2:])


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("order", ["out_in", "in_out"])
def test_grouped_experts_apart_by_any_stride(T, order):
    """Expert matrices that neither touch nor lie a whole number of rows apart."""
    E, K, N_ = 3, 56, 40
    a, b = (N_, K) if order == "out_in" else (K, N_)
    flat = torch.full((E * (a * 72 + 8),), float("nan"), dtype=BF, device="cuda")
    w = flat.as_strided((E, a, b), (a * 72 + 8, 72, 1))
    w.copy_(torch.randn(E, a, b, generator=_gen(7), device="cuda") * 0.05)
    x = torch.randn(T, K, generator=_gen(8), device="cuda").to(BF)
    off = torch.tensor([0, 1, 1, T], dtype=torch.int32, device="cuda")
    _run_dense(moe.GroupedExperts(w, order=order), T, 1, N_, False, False, off, None, x, w, None, order, F32)


@pytest.mark.parametrize("T", [2, 300])
def test_grouped_expert_stride_past_32_bits(T):
    """The second expert lies more than 2^32 bytes (and 2^31 elements) behind the first."""
    E, K, N_ = 2, 64, 40
    stride = (1 << 31) + 64
    flat = torch.empty(stride + N_ * K, dtype=BF, device="cuda")
    w = flat.as_strided((E, N_, K), (stride, K, 1))
    w.copy_(torch.randn(E, N_, K, generator=_gen(3), device="cuda") * 0.05)
    x = torch.randn(T, K, generator=_gen(4), device="cuda").to(BF)
    off = torch.tensor([0, 1, T], dtype=torch.int32, device="cuda")
    _run_dense(moe.GroupedExperts(w), T, 1, N_, False, False, off, None, x, w, None, "out_in", F32)


@pytest.mark.parametrize("T", [3, 260])
def test_products_captured_replayed_and_on_two_streams(T):
    """Capture on a side stream, replay on changed inputs, and two calls at once: the bits of the eager call."""
    k, E, K, N_ = 2, 6, 192, 96
    _, off, pairs, x, w, w_up = _dense_case(T, k, E, K, N_, True, True, BF, BF, "out_in")
    op = moe.GroupedExperts(w, w_up, y_dtype=BF)
    q, s, z = _quantize(torch.randn(E, N_, K, generator=_gen(9), device="cuda") * 0.05, 64, True)
    four = moe.W4Experts(q, s, z, group=64, x_dtype=BF, y_dtype=F32)
    ref, ref4 = op(x, off, pairs, k=k).clone(), four(x, off, pairs, k=k).clone()
    y, y4 = torch.zeros_like(ref), torch.zeros_like(ref4)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        op(x, off, pairs, k=k, out=y)
        four(x, off, pairs, k=k, out=y4)
    for _ in range(2):
        y.zero_()
        y4.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(y4, ref4)
    x2 = x.flip(0).contiguous()
    ref2, ref24 = op(x2, off, pairs, k=k).clone(), four(x2, off, pairs, k=k).clone()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref2) and torch.equal(y4, ref24)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ya, yb = torch.zeros_like(ref), torch.zeros_like(ref)
    for _ in range(10):
        op(x, off, pairs, k=k, out=ya, stream=a)
        op(x, off, pairs, k=k, out=yb, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(ya, ref2) and torch.equal(yb, ref2)


# ------------------------------------------------------------------ 4-bit weights

def _quantize(w, group, zeros, scale_dtype=HF):
    E, N_, K = w.shape
    v = w.view(E, N_, K // group, group).float()
    if zeros:
        lo, hi = v.amin(3, keepdim=True), v.amax(3, keepdim=True)
        s = ((hi - lo) / 15).to(scale_dtype).float()
        z = (-lo / s).round().clamp(0, 15)
    else:
        s = (v.abs().amax(3, keepdim=True) / 7).to(scale_dtype).float()
        z = torch.full_like(s, 8.0)
    c = (v / s + z).round().clamp(0, 15).to(torch.uint8).view(E, N_, K)
    q = (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()
    return q, s[..., 0].to(scale_dtype).contiguous(), (z[..., 0].to(torch.uint8).contiguous() if zeros else None)


def _dequant(q, s, z, group):
    def one(e):
        c = torch.stack((q[e] & 15, q[e] >> 4), dim=2).double().flatten(1)
        zz = 8.0 if z is None else z[e].double().repeat_interleave(group, 1)
        return (c - zz) * s[e].double().repeat_interleave(group, 1)
    return one


_FOUR = [
    # T, k, E, K, N, up, gather, x dtype, y dtype, group, zeros, scale dtype, pad
    (1, 1, 1, 32, 1, False, False, BF, F32, 32, False, HF, 0),
    (1, 1, 1, 64, 17, True, False, HF, F32, 64, True, BF, 8),
    (1, 8, 128, 256, 96, True, True, BF, BF, 128, False, HF, 0),
    (2, 2, 4, 96, 33, False, True, HF, HF, 32, True, HF, 8),
    (9, 2, 3, 320, 65, True, True, BF, F32, 64, False, BF, 16),
    (17, 1, 2, 384, 64, False, False, BF, F32, 128, True, HF, 0),
    (33, 3, 5, 1120, 70, True, True, HF, HF, 32, True, HF, 8),
    (100, 2, 3, 640, 40, True, False, BF, BF, 128, True, HF, 0),
    (50, 1, 1, 2048, 48, False, False, HF, F32, 32, False, BF, 0),
    (5, 2, 1024, 64, 16, False, True, BF, F32, 64, True, HF, 0),
]


@pytest.mark.parametrize("case", _FOUR, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_w4_products(case):
    T, k, E, K, N_, up, gather, dtype, y_dtype, group, zeros, s_dtype, pad = case
    gen = _gen(len(str(case)))
    off, pairs = _routing(_split(T * k, E, K), T, k, gen)
    x = _padded(T if gather else T * k, K, pad, dtype, gen, fill=float("nan"))
    rand = lambda: torch.randn(E, N_, K, generator=gen, device="cuda") * 0.05  # noqa: E731
    a = _quantize(rand(), group, zeros, s_dtype)
    b = _quantize(rand(), group, zeros, s_dtype) if up else None
    op = moe.W4Experts(*a, up=b, group=group, x_dtype=dtype, y_dtype=y_dtype)
    full = torch.full((T * k, N_ + 3), 7.0, dtype=y_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    op(x, off, pairs if gather else None, k=k, out=full[:, :N_], status=status)
    torch.cuda.synchronize()
    assert status.item() == N.MOE_OK
    o = off.tolist()
    g, ga, u, ua = _expected(x, _dequant(*a, group), _dequant(*b, group) if up else None, o, _rows_of(gather, o, pairs, k))
    assert bool((full[:, N_:] == 7.0).all()) and bool((full[o[-1]:] == 7.0).all())
    want, tol = _finish(g, ga, u, ua, K // 16 + K // group + 40)
    _close(full[: o[-1], :N_], want, tol, y_dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_every_code_and_zero_point_is_exact(dtype, group):
    """x picks out single weights: each output is one scale * (code - zero), with no rounding at all."""
    N_, K = 16, 256
    code = (torch.arange(N_ * K).view(N_, K) * 7 + torch.arange(N_).view(N_, 1)) % 16
    zero = (torch.arange(N_ * K // group).view(N_, -1) * 5) % 16
    scale = 2.0 ** (torch.arange(N_ * K // group).view(N_, -1) % 8 - 4).float()
    q = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    op = moe.W4Experts(q[None].cuda(), scale[None].to(HF).cuda(), zero[None].to(torch.uint8).cuda(), group=group,
                       x_dtype=dtype)
    y = op(torch.eye(K, dtype=dtype, device="cuda"))
    want = (code - zero.repeat_interleave(group, 1)).double() * scale.double().repeat_interleave(group, 1)
    assert torch.equal(y.double().cpu(), want.t())


@pytest.mark.parametrize("T", [3, 20])
def test_w4_bad_routing_is_reported(T):
    """Offsets and pairs outside their range are clamped and reported; nothing is read or written out of range."""
    k, E, K, N_ = 2, 3, 256, 40
    q = _quantize(torch.randn(E, N_, K, generator=_gen(6), device="cuda") * 0.05, 128, True)
    op = moe.W4Experts(*q, group=128)
    off, pairs = _routing([T, T, 0], T, k, _gen(1))
    x = torch.randn(T, K, generator=_gen(2), device="cuda").to(BF)
    good = op(x, off, pairs, k=k).clone()
    for which in ("offset above", "offset below", "pair above", "pair below"):
        o, p = off.clone(), pairs.clone()
        if which == "offset above":
            o[3] = 2 * T + 5
        elif which == "offset below":
            o[0] = -3
        else:
            p[1] = 2 * T if which == "pair above" else -1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = op(x, o, p, k=k, status=status)
        torch.cuda.synchronize()
        assert status.item() == N.MOE_ERR_DEVICE_CHECK, which
        keep = torch.ones(2 * T, dtype=torch.bool, device="cuda")
        if which.startswith("pair"):
            keep[1] = False
        assert torch.equal(y[keep], good[keep]), which


@pytest.mark.parametrize("offset", [1, 2, 8])
def test_w4_scales_and_zero_points_at_any_place(offset):
    """Scales and zero points that start on their element only (the fast copies need more)."""
    E, N_, K, T = 2, 33, 512, 4
    for group in (32, 64, 128):
        q, s, z = _quantize(torch.randn(E, N_, K, generator=_gen(group), device="cuda") * 0.05, group, True)
        x = torch.randn(T, K, generator=_gen(3), device="cuda").to(HF)
        off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
        ref = moe.W4Experts(q, s, z, group=group, x_dtype=HF)(x, off)
        s2 = torch.empty(s.numel() + offset, dtype=HF, device="cuda")[offset:].view(s.shape).copy_(s)
        z2 = torch.empty(z.numel() + offset, dtype=torch.uint8, device="cuda")[offset:].view(z.shape).copy_(z)
        assert torch.equal(moe.W4Experts(q, s2, z2, group=group, x_dtype=HF)(x, off), ref)


def test_w4_nan_and_inf_stay_in_their_row():
    E, N_, K, T = 2, 40, 128, 6
    q, s, z = _quantize(torch.randn(E, N_, K, generator=_gen(1), device="cuda") * 0.05, 32, True)
    x = torch.randn(T, K, generator=_gen(2), device="cuda").to(BF)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    op = moe.W4Experts(q, s, z, group=32)
    good = op(x, off).clone()
    x[1, 3] = float("nan")
    s[1, 7, 2] = float("inf")
    bad = op(x, off)
    assert bool(torch.isnan(bad[1]).all()) and torch.equal(bad[[0, 2]], good[[0, 2]])
    assert not bool(torch.isfinite(bad[3:, 7]).any())
    cols = [c for c in range(N_) if c != 7]
    assert torch.equal(bad[3:, cols], good[3:, cols])


@pytest.mark.parametrize("gather", [False, True])
def test_grouped_wait_that_runs_out_is_reported(gather):
    """The test setting's stalled wait: the call returns, says so, and the next call gives the bits of the one before."""
    T, k, E, K, N_ = 200, 2, 3, 1024, 300
    _, off, pairs, x, w, _ = _dense_case(T, k, E, K, N_, False, gather, BF, F32, "out_in")
    op = moe.GroupedExperts(w)
    assert op.path(T, k) == "tensor"
    p = pairs if gather else None
    ref = op(x, off, p, k=k).clone()
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        N.moe_debug_set_waits(2_000_000, 1)
        op(x, off, p, k=k, status=status)
        torch.cuda.synchronize()
    finally:
        N.moe_debug_set_waits(0, 0)
    assert status.item() == N.MOE_ERR_TIMEOUT
    assert torch.equal(op(x, off, p, k=k), ref)


@pytest.mark.parametrize("K", [128, 32768])
def test_w4_longest_and_shortest_rows(K):
    """The longest n_in leaves room for one staged row at a time; rows of 128 are half a stage."""
    E, N_, T = 2, 70, 5
    gen = _gen(K)
    a = _quantize(torch.randn(E, N_, K, generator=gen, device="cuda") * 0.02, 32, True)
    x = torch.randn(T, K, generator=gen, device="cuda").to(BF)
    off = torch.tensor([0, 4, 5], dtype=torch.int32, device="cuda")
    y = moe.W4Experts(*a, group=32)(x, off)
    g, ga, _, _ = _expected(x, _dequant(*a, 32), None, off.tolist(), torch.arange(T, device="cuda"))
    want, tol = _finish(g, ga, None, None, K // 16 + K // 32 + 40)
    _close(y, want, tol, F32)


def test_w4_rows_of_very_different_magnitudes():
    """Rows of x are scaled one by one: from 2^-100 to 2^100, and one of zeros."""
    E, N_, K = 1, 48, 256
    gen = _gen(21)
    a = _quantize(torch.randn(E, N_, K, generator=gen, device="cuda") * 0.02, 64, True)
    x = torch.randn(6, K, generator=gen, device="cuda")
    x *= torch.tensor([2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** 100, 0.0], device="cuda")[:, None]
    x = x.to(BF)
    y = moe.W4Experts(*a, group=64)(x)
    g, ga, _, _ = _expected(x, _dequant(*a, 64), None, [0, 6], torch.arange(6, device="cuda"))
    want, tol = _finish(g, ga, None, None, K // 16 + K // 64 + 40)
    _close(y, want, tol, F32)
    assert bool((y[5] == 0).all())


def test_w4_wait_that_runs_out_is_reported():
    T, E, K, N_ = 3, 4, 512, 200
    a = _quantize(torch.randn(E, N_, K, generator=_gen(4), device="cuda") * 0.02, 128, False)
    x = torch.randn(T, K, generator=_gen(5), device="cuda").to(BF)
    off = torch.tensor([0, 1, 1, 2, 3], dtype=torch.int32, device="cuda")
    op = moe.W4Experts(*a, group=128)
    ref = op(x, off).clone()
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        N.moe_debug_set_waits(2_000_000, 1)
        op(x, off, status=status)
        torch.cuda.synchronize()
    finally:
        N.moe_debug_set_waits(0, 0)
    assert status.item() == N.MOE_ERR_TIMEOUT
    assert torch.equal(op(x, off), ref)
