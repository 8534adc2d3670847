"""4-bit products whose rows of x are far from a normal distribution: channels far above the others, rows of one sign,
weights equal to their zero points, infinities, tiny rows.

Tolerances, before any run.  A weight scale * (q - z) is exact as an operand, so the error is that of the sums alone: per
element as test_gpu_products states it, |error| <= depth * 2^-23 * sum |w x|, in which a weight equal to its zero point
counts nothing, whatever x is there.  x itself is exact in these cases: fp16 always, bf16 down to 2^-31 of the row's largest.
In norm, for zero-mean weights: at most two chains of 4 instructions a group, each off by half a unit on average, a unit
being at most 2^-23 of the partial sum, which is 2/3 of the chain's on average: 4 * 2^-24 * 2 / 3; the scale, the two
chains, the groups (errors of either sign, up to 224 of them: half a unit times the root of their number, on partial sums that
are 1 / sqrt(2) of the whole in norm: 224 ** 0.5 / sqrt(12) * 2^-23 / sqrt(2)) and the join.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from test_gpu_products import _close, _dequant, _expected, _finish, _quantize, _routing, _split

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _weights(E, N, K, group, zeros, gen, channel=None):
    """A quantized matrix; at `channel` every code is its zero point."""
    q, s, z = _quantize(torch.randn(E, N, K, generator=gen, device="cuda") * 0.05, group, zeros)
    if channel is not None:
        zz = torch.full((E, N), 8, dtype=torch.uint8, device="cuda") if z is None else z[:, :, channel // group]
        byte = q[:, :, channel // 2]
        q[:, :, channel // 2] = (byte & 0xF0) | zz if channel % 2 == 0 else (byte & 0x0F) | (zz << 4)
    return q, s, z


# T, k, E, K, N, up, gather, group, zeros
_CASES = [(8, 1, 1, 128, 256, False, False, 128, False), (1, 2, 3, 2048, 130, True, True, 64, True),
          (3, 2, 4, 320, 70, False, True, 32, True), (16, 2, 3, 1024, 96, True, False, 128, True),
          (40, 1, 2, 7168, 48, False, False, 64, False)]


@pytest.mark.parametrize("case", _CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["channel", "channel of 2^20", "one sign", "both"])
def test_w4_rows_far_from_normal(case, dtype, kind):
    T, k, E, K, N, up, gather, group, zeros = case
    gen = torch.Generator(device="cuda").manual_seed(K + len(kind))
    off, pairs = _routing(_split(T * k, E, K), T, k, gen)
    x = torch.randn(T if gather else T * k, K, generator=gen, device="cuda")
    channel = None
    if kind in ("one sign", "both"):
        x = x.abs()
    if kind != "one sign":
        channel = 2 * (K // 5) + 1
        x[:, channel] = 2.0 ** 20 if kind.endswith("2^20") and dtype is BF else 20000.0
    x = x.to(dtype)
    a = _weights(E, N, K, group, zeros, gen, channel)
    b = _weights(E, N, K, group, zeros, gen, channel) if up else None
    y = moe.W4Experts(*a, up=b, group=group, x_dtype=dtype)(x, off, pairs if gather else None, k=k)
    o = off.tolist()
    rows = (pairs.long() // k) if gather else torch.arange(o[-1], device="cuda")
    g, ga, u, ua = _expected(x, _dequant(*a, group), _dequant(*b, group) if up else None, o, rows)
    want, tol = _finish(g, ga, u, ua, K // 16 + K // group + 40)
    _close(y[: o[-1]], want, tol, F32)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("K, group", [(128, 128), (2048, 64), (7168, 32)])
def test_w4_rows_of_one_sign_keep_their_precision(dtype, K, group):
    gen = torch.Generator(device="cuda").manual_seed(K)
    a = _weights(1, 256, K, group, False, gen)
    x = torch.randn(8, K, generator=gen, device="cuda").abs().to(dtype)
    y = moe.W4Experts(*a, group=group, x_dtype=dtype)(x).double()
    exact = x.double() @ _dequant(*a, group)(0).t()
    bound = 4 * 2.0 ** -24 * 2 / 3 + 224 ** 0.5 / 12 ** 0.5 * 2.0 ** -23 / 2 ** 0.5 + 3 * 2.0 ** -24
    assert ((y - exact).norm() / exact.norm()).item() <= bound


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_w4_weights_equal_to_their_zero_points_give_zero(T, group, zeros):
    gen = torch.Generator(device="cuda").manual_seed(T)
    K, N = 768, 40
    z = torch.randint(0, 16, (1, N, K // group), generator=gen, device="cuda", dtype=torch.uint8)
    if not zeros:
        z.fill_(8)
    c = z.repeat_interleave(group, 2)
    q = c[..., 0::2] | (c[..., 1::2] << 4)
    s = torch.rand(1, N, K // group, generator=gen, device="cuda").half()
    x = (torch.randn(T, K, generator=gen, device="cuda") * 100).bfloat16()
    assert bool((moe.W4Experts(q, s, z if zeros else None, group=group)(x) == 0).all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_w4_infinities_give_the_formula_s_values(dtype):
    """An infinity times q - z: infinite with its sign, NaN for 0; the row's other values do not matter."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    K, N, group = 256, 64, 64
    a = _weights(1, N, K, group, True, gen)
    x = (torch.randn(4, K, generator=gen, device="cuda") * (1e30 if dtype is BF else 6e3)).to(dtype)
    x[1, 7], x[2, 100] = float("inf"), float("-inf")
    y = moe.W4Experts(*a, group=group, x_dtype=dtype)(x).double()
    w = _dequant(*a, group)(0)
    assert bool((w[:, 7] == 0).any()) and bool((w[:, 7] != 0).any())
    for r, c in ((1, 7), (2, 100)):
        want = x[r, c].double() * w[:, c]
        assert torch.equal(torch.nan_to_num(y[r], nan=5.0), torch.nan_to_num(want, nan=5.0))
    assert bool(torch.isfinite(y[[0, 3]]).all())


def test_w4_rows_of_subnormal_numbers():
    gen = torch.Generator(device="cuda").manual_seed(2)
    K, N, group = 256, 64, 64
    a = _weights(1, N, K, group, False, gen)
    x = (torch.randint(-100, 101, (3, K), generator=gen, device="cuda").double() * 2.0 ** -133).to(BF)
    assert bool((x.double().abs().amax(1) > 0).all()) and x.double().abs().max().item() < 2.0 ** -126
    y = moe.W4Experts(*a, group=group)(x)
    g, ga, _, _ = _expected(x, _dequant(*a, group), None, [0, 3], torch.arange(3, device="cuda"))
    want, tol = _finish(g, ga, None, None, K // 16 + K // group + 40)
    _close(y, want, tol, F32)
