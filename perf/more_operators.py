"""Operators around the routed experts: what is measured, the plain forms and the exact values.

  linear    y = res_scale * residual + scale * act(x W^T + bias) over bf16 or fp16 weights
  norm_fwd  layer norm: y, and each row's mean and reciprocal deviation
  norm_bwd  its gradient: dx (added to the residual stream's), and the sums over the rows for gamma and beta
  balance   the router's balance loss over the logits and the chosen experts, counts per expert, and its gradient

A case is a dict of plain values; prepare() makes what a program holds before the call, run() makes one call.
"""
import math

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
_DT = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
_SIZE = {BF16: 2, F16: 2, F32: 4}
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _linear(name, T, K, N, x=BF16, y=BF16, act="none", bias="f32", res=None, order="out_in", pad=0):
    return dict(name=name, op="linear", T=T, K=K, N=N, x=x, y=y, act=act, bias=bias or "", res=res or "", order=order, pad=pad)


def _norm(name, op, T, H, x=F32, y=BF16, add=False, pad=0):
    return dict(name=name, op=op, T=T, H=H, x=x, y=y, add=add, pad=pad)


def _balance(name, T, E, k, mode="softmax", seqs=0, mask=False, grad=True, pad=0):
    return dict(name=name, op="balance", T=T, E=E, k=k, mode=mode, seqs=seqs, mask=mask, grad=grad, pad=pad)


def listed():
    return [
        # one decoded token through a square projection that adds to the fp32 residual stream (hidden 2048)
        _linear("linear T1 residual", 1, 2048, 2048, y=F32, res=F32),
        # a decode batch of 32 through the down half of a dense block of the large model (7168 -> 2048)
        _linear("linear T32 gelu", 32, 7168, 2048, act="gelu"),
        # a prompt of 4096 tokens: the up half of a dense block, with its activation
        _linear("linear T4096 gelu", 4096, 2048, 7168, act="gelu"),
        # the same prompt: the down half, added to the fp32 residual stream
        _linear("linear T4096 residual", 4096, 7168, 2048, y=F32, res=F32),
        # odd sizes, padded rows, fp16, weights stored [in][out]: no dimension a multiple of a tile
        _linear("linear odd f16", 301, 1000, 1333, x=F16, y=F16, act="silu", bias="f16", res=F16, order="in_out", pad=24),
        # one decoded token in front of a block
        _norm("norm forward T1", "norm_fwd", 1, 2048),
        # a prompt of 4096 tokens, fp32 residual stream
        _norm("norm forward T4096", "norm_fwd", 4096, 2048),
        # training over 4096 tokens: the gradient through the norm joins that of the residual stream
        _norm("norm backward T4096", "norm_bwd", 4096, 2048, add=True),
        # a small batch of the large model, bf16 stream, padded rows
        _norm("norm backward T512 bf16", "norm_bwd", 512, 7168, x=BF16, pad=8),
        # a decode batch of 32 over 128 experts: loss and counts, as a monitor and with its gradient
        _balance("balance T32", 32, 128, 8),
        # a training batch of 4096 tokens, padded places masked
        _balance("balance T4096", 4096, 128, 8, mask=True),
        # 16 packed sequences of uneven length over 256 experts, sigmoid scores, rows behind the last sequence
        _balance("balance T32768 sequences", 32768, 256, 8, mode="sigmoid", seqs=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "norm_fwd", "norm_bwd", "balance"))
    if op == "linear":
        while True:
            T, K, N = _log_int(rng, 1, 8192), _log_int(rng, 16, 16384), _log_int(rng, 16, 16384)
            if rng.random() < 0.5:
                K, N = 8 * (K // 8), 8 * (N // 8)
            if T * K * N <= 60e9 and K * N <= 60e6 and T * (K + N) <= 36e6:
                x = rng.choice((BF16, F16))
                return dict(op=op, T=T, K=K, N=N, x=x, y=rng.choice((F32, x)), act=rng.choice(_ACTS),
                            bias=rng.choice(("", "f32", x)), res=rng.choice(("", F32, x)),
                            order=rng.choice(("out_in", "in_out")), pad=rng.choice((0, 0, 8, 24)))
    if op == "balance":
        E = rng.choice((_log_int(rng, 4, 512), 32 * rng.randint(1, 12)))
        T = min(_log_int(rng, 1, 32768), (1 << 23) // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 8)), mode=rng.choice(("softmax", "sigmoid")),
                    seqs=rng.choice((0, 0, 1, _log_int(rng, 2, 64))), mask=rng.random() < 0.4, grad=rng.random() < 0.8,
                    pad=rng.choice((0, 0, 4, 3)))
    H = rng.choice((_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)))
    T = max(1, min(_log_int(rng, 1, 4096), (1 << 23) // H))
    return dict(op=op, T=T, H=H, x=rng.choice((F32, BF16, F16)), y=rng.choice((F32, BF16, F16)),
                add=op == "norm_bwd" and rng.random() < 0.5, pad=rng.choice((0, 0, 8, 3)))


# ------------------------------------------------------------------ inputs

def _rows(gen, n, width, pad, dtype, scale=1.0):
    """[n, width] values in rows of width + pad elements."""
    return torch.empty(n, width + pad, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1 + seed)
    s = dict(case=case)
    T, pad = case["T"], case["pad"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        dt = _DT[case["x"]]
        s["x"] = _rows(gen, T, K, -K % 8 + pad, dt)
        a, b = (N, K) if case["order"] == "out_in" else (K, N)
        s["w"] = _rows(gen, a, b, -b % 8, dt, 1.0 / math.sqrt(K))
        s["bias"] = torch.empty(N, dtype=_DT[case["bias"]], device="cuda").normal_(0.0, 0.5, generator=gen) if case["bias"] else None
        s["res"] = _rows(gen, T, N, pad, _DT[case["res"]], 2.0) if case["res"] else None
        s["scale"], s["res_scale"] = (1.25, 0.5) if case["res"] else (1.0, 1.0)
        s["out"] = torch.empty(T, N + pad, dtype=_DT[case["y"]], device="cuda")[:, :N]
        if own:
            import quantized_routed_expert_sigmoid_gb300 as moe
            s["op"] = moe.Linear(s["w"], s["bias"], order=case["order"], act=case["act"], y_dtype=_DT[case["y"]],
                                 scale=s["scale"], res_scale=s["res_scale"])
        return s
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        popular = torch.empty(E, device="cuda").normal_(0.0, 0.7, generator=gen)
        s["logits"] = _rows(gen, T, E, pad, torch.float32)
        s["logits"] += popular
        s["ids"] = torch.topk(s["logits"], k, dim=1).indices.sort(dim=1).values.to(torch.int32)
        s["mask"] = torch.rand(T, device="cuda", generator=gen) < 0.9 if case["mask"] else None
        s["offsets"] = None
        if case["seqs"]:
            # uneven lengths (some may be empty), a few rows behind the last sequence
            cut = torch.rand(case["seqs"] + 1, device="cuda", generator=gen)
            cut = torch.sort(cut).values * T
            cut[0] = 0
            s["offsets"] = cut.to(torch.int32)
        s["upstream"] = torch.full((1,), 1.5, device="cuda")
        s["coef"] = 0.01
        if own:
            import quantized_routed_expert_sigmoid_gb300 as moe
            s["op"] = moe.BalanceLoss(E, k, mode=case["mode"], coef=s["coef"])
            s["dlogits"] = torch.empty(T, E, device="cuda") if case["grad"] else None
        return s
    H = case["H"]
    s["gamma"] = 1.0 + torch.empty(H, device="cuda").normal_(0.0, 0.1, generator=gen)
    s["beta"] = torch.empty(H, device="cuda").normal_(0.0, 0.1, generator=gen)
    s["eps"] = 1e-5
    s["x"] = _rows(gen, T, H, pad, _DT[case["x"]], 2.0)
    s["x"] += 0.5
    if case["op"] == "norm_bwd":
        s["dy"] = _rows(gen, T, H, pad, _DT[case["y"]])
        s["add"] = _rows(gen, T, H, pad, _DT[case["x"]]) if case["add"] else None
        x = s["x"].double()
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = (1.0 / ((x - mean[:, None]).pow(2).mean(1) + s["eps"]).sqrt()).float()
    if own:
        import quantized_routed_expert_sigmoid_gb300 as moe
        s["op"] = moe.LayerNorm(H, gamma=s["gamma"], beta=s["beta"], eps=s["eps"])
        s["out"] = torch.empty(T, H, dtype=_DT[case["y" if case["op"] == "norm_fwd" else "x"]], device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return {"linear": _plain_linear, "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_backward,
                "balance": _plain_balance}[case["op"]](s)
    if case["op"] == "linear":
        return s["op"](s["x"], residual=s["res"], out=s["out"])
    if case["op"] == "norm_fwd":
        return list(s["op"](s["x"], out=s["out"]))
    if case["op"] == "norm_bwd":
        return list(s["op"].backward(s["dy"], s["x"], s["mean"], s["rstd"], add=s["add"], dx=s["out"]))
    loss, counts, dlogits = s["op"](s["logits"], s["ids"], offsets=s["offsets"], mask=s["mask"], dlogits=s["dlogits"],
                                    upstream=s["upstream"])
    return [loss, counts] + ([dlogits] if case["grad"] else [])


def _plain_linear(s):
    case, w = s["case"], s["w"].float()
    z = s["x"].float() @ (w.t() if case["order"] == "out_in" else w)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    act = case["act"]
    if act == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif act == "gelu":
        z = 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    elif act == "gelu_tanh":
        z = z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    z = s["scale"] * z
    if s["res"] is not None:
        z = z + s["res_scale"] * s["res"].float()
    return z.to(_DT[case["y"]])


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["gamma"] + s["beta"]
    return [y.to(_DT[s["case"]["y"]]), mean[:, 0], rstd[:, 0]]


def _plain_norm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return [dx.to(_DT[s["case"]["x"]]), (dy * xh).sum(0), dy.sum(0)]


def _plain_balance(s):
    case, logits = s["case"], s["logits"]
    T, E, k, B = case["T"], case["E"], case["k"], max(case["seqs"], 1)
    if s["offsets"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device="cuda")
    else:
        t = torch.arange(T, device="cuda")
        seq = (t[:, None] >= s["offsets"][None, 1:]).sum(1)          # B: behind the last sequence
    live = seq < B
    if s["mask"] is not None:
        live = live & s["mask"]
    at = torch.where(live, seq, torch.full_like(seq, B))
    n = torch.zeros(B + 1, device="cuda").index_add_(0, at, torch.ones(T, device="cuda"))[:B]
    counts = torch.zeros((B + 1) * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, (at[:, None] * E + s["ids"].long()).reshape(-1), torch.ones(T * k, dtype=torch.int32, device="cuda"))
    counts = counts.view(B + 1, E)[:B]
    if case["mode"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p, slope = e / e.sum(1, keepdim=True), 1.0
    else:
        sig = 1.0 / (1.0 + torch.exp(-logits))
        p, slope = sig / sig.sum(1, keepdim=True), 1.0 - sig
    P = torch.zeros(B + 1, E, dtype=torch.float64, device="cuda").index_add_(0, at, p.double())[:B].float()   # (a long sum)
    some = (n > 0).float()
    per = some / torch.clamp(n, min=1.0)
    f = counts.float() * (E / k) * per[:, None]
    coef = s["coef"] / torch.clamp(some.sum(), min=1.0)
    loss = coef * (f * P * per[:, None]).sum()
    out = [loss.reshape(1), counts]
    if case["grad"]:
        b = torch.clamp(at, max=B - 1)
        ft = f[b]
        g = p * (ft - (ft * p).sum(1, keepdim=True)) * slope
        out.append(torch.where(live[:, None], g * (coef * s["upstream"] * per[b])[:, None], torch.zeros_like(g)))
    return out


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "linear":
        if case["order"] == "out_in":
            z = torch.einsum("tc,nc->tn", s["x"].double(), s["w"].double())
        else:
            z = torch.einsum("tc,cn->tn", s["x"].double(), s["w"].double())
        z = z if s["bias"] is None else z + s["bias"].double()
        act = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0.0),
               "gelu": lambda v: v * torch.special.ndtr(v),
               "gelu_tanh": lambda v: 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))),
               "silu": lambda v: v * torch.sigmoid(v)}[case["act"]]
        z = act(z) * s["scale"]
        return z if s["res"] is None else z + s["res"].double() * s["res_scale"]
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        off = [0, T] if s["offsets"] is None else s["offsets"].tolist()
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        rows = [(a + keep[a:b].nonzero()[:, 0]) for a, b in zip(off[:-1], off[1:])]
        used = sum(len(r) > 0 for r in rows)
        loss = torch.zeros((), dtype=torch.float64, device="cuda")
        counts = torch.zeros(len(rows), E, dtype=torch.int32, device="cuda")
        grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        for b, r in enumerate(rows):
            n = len(r)
            if n == 0:
                continue
            v = s["logits"][r].double()
            score = torch.softmax(v, 1) if case["mode"] == "softmax" else torch.sigmoid(v)
            p = score / score.sum(1, keepdim=True)
            counts[b] = torch.bincount(s["ids"][r].reshape(-1).long(), minlength=E)
            w = counts[b].double() * (E / (k * n)) * (s["coef"] / (used * n))       # dL/dp
            loss += (w * p.sum(0)).sum()
            down = p * (w - (p @ w)[:, None])
            grad[r] = down * 1.5 if case["mode"] == "softmax" else down * torch.sigmoid(-v) * 1.5
        return [loss.reshape(1), counts] + ([grad] if case["grad"] else [])
    x = s["x"].double()
    H = case["H"]
    if case["op"] == "norm_fwd":
        mean = x.sum(1) / H
        var = (x - mean.unsqueeze(1)).square().sum(1) / H
        rstd = (var + s["eps"]).rsqrt()
        return [torch.addcmul(s["beta"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["gamma"].double()), mean, rstd]
    # the gradient at the row's own mean and deviation
    mean = x.sum(1, keepdim=True) / H
    xh = x - mean
    rstd = (xh.square().sum(1, keepdim=True) / H + s["eps"]).rsqrt()
    xh = xh * rstd
    dy = s["dy"].double()
    g = dy * s["gamma"].double()
    dx = (g - (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True)) / H) * rstd
    if s["add"] is not None:
        dx = dx + s["add"].double()
    return [dx, torch.einsum("th,th->h", dy, xh), dy.sum(0)]


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        per = _SIZE[case["y"]] + (_SIZE[case["res"]] if case["res"] else 0)
        return {"bytes": 2 * (N * K + T * K) + T * N * per + (N * _SIZE[case["bias"]] if case["bias"] else 0),
                "flops": 2.0 * T * N * K}
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        B = max(case["seqs"], 1)
        return {"bytes": 4 * T * E * (2 if case["grad"] else 1) + 4 * T * k + 4 * B * E + (T if case["mask"] else 0),
                "flops": 12.0 * T * E}
    H, x, y = case["H"], _SIZE[case["x"]], _SIZE[case["y"]]
    if case["op"] == "norm_fwd":
        return {"bytes": T * H * (x + y) + 8 * T + 8 * H, "flops": 8.0 * T * H}
    return {"bytes": T * H * (x * (3 if case["add"] else 2) + y) + 8 * T + 12 * H, "flops": 16.0 * T * H}
