"""Layer norm, dense products, the router and its balance loss as the parts of a block around the routed experts:

  u = norm(x); h = gelu(u W1^T + b1); x1 = x + h W2^T + b2; v = norm(x1); route v; loss and its gradient;
  the gradient through the second norm, joined with the residual stream's

Each step is checked against its formula in 64 bits on the values that the step before it gave, with the tolerances of the
operators' own tests.
"""
from __future__ import annotations

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from quantized_routed_expert_sigmoid_gb300 import _native as N
import test_gpu_balance as tb
import test_gpu_layer_norm as tn
import test_gpu_linear as tl

pytestmark = pytest.mark.gpu

BF, F32, U = torch.bfloat16, torch.float32, 2.0 ** -24


class Block:
    def __init__(self, H=512, F=1280, E=32, k=4):
        g = torch.Generator(device="cuda").manual_seed(3)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.H, self.E, self.k = H, E, k
        self.w1, self.w2 = (rand(F, H) / H ** 0.5).to(BF), (rand(F, H) / F ** 0.5).to(BF)      # w2 stored [in][out]
        self.b1, self.b2 = rand(F), rand(H).to(BF)
        self.g1, self.g2, self.c1, self.c2 = (s + 0.1 * rand(H) for s in (1, 1, 0, 0))
        self.Wr = rand(E, H) * 0.05
        self.norm1, self.norm2 = moe.LayerNorm(H, gamma=self.g1, beta=self.c1), moe.LayerNorm(H, gamma=self.g2, beta=self.c2)
        self.up = moe.Linear(self.w1, self.b1, act="gelu")
        self.down = moe.Linear(self.w2, self.b2, order="in_out", y_dtype=F32, scale=0.5)
        self.cfg = moe.route_cfg(moe.MOE_ROUTE_SOFTMAX, E, k)
        self.balance = moe.BalanceLoss(E, k, coef=0.01)

    def run(self, x, off, dv, dx1, s=None):
        T = x.shape[0]
        with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
            logits, ids = torch.empty(T, self.E, device="cuda"), torch.empty(T, self.k, dtype=torch.int32, device="cuda")
            gates = torch.empty(T, self.k, device="cuda")
        u, _, _ = self.norm1(x, stats=False, stream=s)
        h = self.up(u, stream=s)
        x1 = self.down(h, residual=x, stream=s)
        v, mean, rstd = self.norm2(x1, stream=s)
        moe.moe_route(self.cfg, v, moe.MOE_BF16, T, self.H, self.Wr, None, None, logits, ids, gates, stream=s)
        loss, counts, dlogits = self.balance(logits, ids, offsets=off, dlogits=True, stream=s)
        dx, dg, db = self.norm2.backward(dv, x1, mean, rstd, add=dx1, stream=s)
        return [u, h, x1, v, mean, rstd, logits, ids, loss, counts, dlogits, dx, dg, db]

    def check(self, x, off, dv, dx1, got):
        u, h, x1, v, mean, rstd, logits, ids, loss, counts, dlogits, dx, dg, db = got

        def norm(y, x, g, c):
            m, q, xh, e = tn._stats(x, 1e-5)
            want = xh * g.double() + c.double()
            tn._close(y, want, e * g.double().abs() + U * ((xh * g.double()).abs() + want.abs()))
            return xh, e, q

        norm(u, x, self.g1, self.c1)
        tl._close(h, *tl._want(u, self.w1, "out_in", self.b1, "gelu", 1.0, None, 1.0, BF))
        tl._close(x1, *tl._want(h, self.w2, "in_out", self.b2, "none", 0.5, x, 1.0, F32))
        xh, e, q = norm(v, x1, self.g2, self.c2)
        tb._compare((loss, counts, dlogits), tb._want(logits, ids, self.k, "softmax", 0.01, off.tolist()))
        g = dv.double() * self.g2.double()
        want = dx1.double() + q * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        a, b, c = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True), (g.abs() * e).mean(1, keepdim=True)
        tn._close(dx, want, q * (48 * U * (g.abs() + a + xh.abs() * b) + xh.abs() * c + e * b) + U * (dx1.double().abs() + want.abs()))
        depth = U * (x.shape[0] / 150 + 66)
        tn._close(dg, (dv.double() * xh).sum(0), depth * (dv.double() * xh).abs().sum(0) + (dv.double().abs() * e).sum(0))
        tn._close(db, dv.double().sum(0), depth * dv.double().abs().sum(0))


@pytest.mark.parametrize("T", [1, 7, 64, 300, 2500])
def test_block_of_the_operators_around_the_experts(T):
    blk = Block()
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dx1 = (torch.randn(T, blk.H, generator=gen, device="cuda") for _ in range(2))
    dv = torch.randn(T, blk.H, generator=gen, device="cuda").to(BF)
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    first = blk.run(x, off, dv, dx1)
    torch.cuda.synchronize()
    blk.check(x, off, dv, dx1, first)
    bits = [t.clone() for t in first]
    # the block captured twice, replayed beside one another and beside an eager one on a stream of its own: the same bits
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            outs.append(blk.run(x, off, dv, dx1))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = blk.run(x, off, dv, dx1, streams[2])
        torch.cuda.synchronize()
        for got in outs + [eager]:
            assert all(torch.equal(a, b) for a, b in zip(got, bits))
    # new inputs in the captured places
    x.copy_(torch.randn(T, blk.H, generator=gen, device="cuda"))
    graphs[0].replay()
    torch.cuda.synchronize()
    blk.check(x, off, dv, dx1, outs[0])
    assert blk.up.device_status() == blk.down.device_status() == blk.balance.device_status() == N.MOE_OK
