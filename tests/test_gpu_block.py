"""The new operators as one block of a stack, next to the layer's own calls, against the formula in 64 bits:

  u = norm(x);  route, permute;  h = silu(Wg u) * (Wu u);  y = Wd h;  combine;  x' = a x + s * norm(y), u' = norm(x')

with unquantized experts (moe_grouped_matmul) and with 4-bit ones (moe_w4_matmul).  Routing ids and gates are the
GPU's own (tested against the oracle elsewhere).  Tolerances, before any run: h is stored in bf16, so its elements are off
by at most 2^-8 relative, independently of each other, and so is the combined y in its 2-norm; everything else on the
way is fp32 (1e-5 at these sizes).  y's norm keeps relative errors, so x' is off by 2^-8 of the normed part and u'
by that and its own bf16 rounding: 2^-8 + 2^-8.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _quantize(w, group):
    E, N_, K = w.shape
    v = w.view(E, N_, K // group, group)
    lo, hi = v.amin(3, keepdim=True), v.amax(3, keepdim=True)
    s = ((hi - lo) / 15).half().float()
    z = (-lo / s).round().clamp(0, 15)
    c = (v / s + z).round().clamp(0, 15).to(torch.uint8).view(E, N_, K)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s[..., 0].half().contiguous(), z[..., 0].to(torch.uint8).contiguous()


def _dequant(q, s, z, group):
    c = torch.stack((q & 15, q >> 4), dim=3).double().flatten(2)
    return (c - z.double().repeat_interleave(group, 2)) * s.double().repeat_interleave(group, 2)


class Block:
    def __init__(self, four, E=16, k=4, H=512, I=256):
        g = torch.Generator(device="cuda").manual_seed(11)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.E, self.k, self.H, self.I, self.four = E, k, H, I, four
        self.Wr = rand(E, H) * 0.05
        self.g0, self.g1, self.g2 = (1 + 0.1 * rand(H) for _ in range(3))
        w = [rand(E, I, H) * 0.05, rand(E, I, H) * 0.05, rand(E, H, I) * 0.05]
        if four:
            q = [_quantize(m, 64) for m in w]
            self.w64 = [_dequant(*m, 64) for m in q]
            self.gate_up = moe.W4Experts(*q[0], up=q[1], group=64, y_dtype=BF)
            self.down = moe.W4Experts(*q[2], group=64)
        else:
            w = [m.to(BF) for m in w]
            self.w64 = [m.double() for m in w]
            self.gate_up = moe.GroupedExperts(w[0], w[1], y_dtype=BF)
            self.down = moe.GroupedExperts(w[2])
        self.norm = moe.NormResidual(H, gamma_post=self.g1, gamma_pre=self.g2, res_scale=0.5, scale=1.5)
        self.cfg = moe.route_cfg(moe.MOE_ROUTE_SOFTMAX, E, k)

    def buffers(self, T):
        P, dev = T * self.k, "cuda"
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
        ws = moe.moe_permute_workspace_size(T, self.k, self.E)
        return dict(u=torch.empty(T, self.H, dtype=BF, device=dev), logits=torch.empty(T, self.E, device=dev), ids=i32(P),
                    gates=torch.empty(P, device=dev), sorted=i32(P), off=i32(self.E + 1), pos=i32(P),
                    ws=torch.empty(ws, dtype=torch.uint8, device=dev), h=torch.empty(P, self.I, dtype=BF, device=dev),
                    y=torch.empty(P, self.H, device=dev), out=torch.empty(T, self.H, device=dev),
                    x_out=torch.empty(T, self.H, device=dev), u_out=torch.empty(T, self.H, dtype=BF, device=dev))

    def run(self, x, b):
        T, k, E, H = x.shape[0], self.k, self.E, self.H
        moe.moe_rmsnorm_bf16(x, self.g0, T, H, 1e-6, b["u"])
        moe.moe_route(self.cfg, b["u"], moe.MOE_BF16, T, H, self.Wr, None, None, b["logits"], b["ids"], b["gates"])
        moe.moe_permute(b["ids"], T, k, E, b["sorted"], b["off"], b["pos"], b["ws"], b["ws"].numel())
        self.gate_up(b["u"], b["off"], b["sorted"], k=k, out=b["h"])
        self.down(b["h"], b["off"], k=k, out=b["y"])
        moe.moe_combine(b["y"], b["gates"], b["pos"], T, k, H, None, 0, b["out"])
        self.norm(x, b["out"], x_out=b["x_out"], u=b["u_out"])

    def expected(self, x, b):
        T, k = x.shape[0], self.k
        u, ids, gates = b["u"].double(), b["ids"].view(T, k).long(), b["gates"].view(T, k).double()
        wg, wu, wd = self.w64
        out = torch.zeros(T, self.H, dtype=torch.float64, device="cuda")
        for j in range(k):
            for e in range(self.E):
                t = (ids[:, j] == e).nonzero()[:, 0]
                if len(t):
                    g = u[t] @ wg[e].t()
                    h = g / (1 + torch.exp(-g)) * (u[t] @ wu[e].t())
                    out[t] += gates[t, j, None] * (h @ wd[e].t())
        n = out / (out.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * self.g1.double()
        r = 0.5 * x.double() + 1.5 * n
        return out, r, r / (r.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * self.g2.double()


def _rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T", [1, 5, 64, 600])
def test_block_of_new_operators(four, T):
    blk = Block(four)
    x = torch.randn(T, blk.H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    b = blk.buffers(T)
    blk.run(x, b)
    torch.cuda.synchronize()
    out, r, u = blk.expected(x, b)
    assert _rel(b["out"], out) <= 2.0 ** -8
    assert _rel(b["x_out"], r) <= 2.0 ** -8
    assert _rel(b["u_out"], u) <= 2.0 ** -7
    # the same block captured: the same bits, on new inputs too, while another block runs eagerly
    bits = b["x_out"].clone(), b["u_out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        blk.run(x, b)
    b["x_out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b["x_out"], bits[0]) and torch.equal(b["u_out"], bits[1])
    x2 = x.flip(1).contiguous()
    c = blk.buffers(T)
    blk.run(x2, c)
    x.copy_(x2)
    graph.replay()
    blk.run(x2, c)
    torch.cuda.synchronize()
    assert torch.equal(b["x_out"], c["x_out"]) and torch.equal(b["u_out"], c["u_out"])
