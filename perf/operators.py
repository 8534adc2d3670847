"""The operators measured here, their plain forms and their exact values.

  grouped   products of the rows of each expert with that expert's bf16 or fp16 weights (ragged sizes), alone or as
            the gated pair silu(W x) * (W_up x), from rows in place or gathered through the routing's pairs
  w4        the same products over 4-bit weights with one scale (and maybe a zero point) per group
  norm      the norm behind a block, its gate and residual scale, and the norm in front of the next block

A case is a dict of plain values; prepare() makes what a program holds before the call, run() makes one call.
"""
import math

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
_DT = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}


def _grouped(name, T, k, E, K, N, up, gather, x="bf16", y="bf16", order="out_in", route="uniform", pad=0):
    return dict(name=name, op="grouped", T=T, k=k, E=E, K=K, N=N, up=up, gather=gather, x=x, y=y, order=order,
                route=route, pad=pad)


def _w4(name, T, k, E, K, N, up, gather, group, zeros, x="bf16", y="bf16"):
    return dict(name=name, op="w4", T=T, k=k, E=E, K=K, N=N, up=up, gather=gather, group=group, zeros=zeros, x=x, y=y,
                route="uniform", pad=0)


def _norm(name, T, H, x="f32", y="f32", u="bf16", post=True, gate="none", pad=0):
    return dict(name=name, op="norm", T=T, H=H, x=x, y=y, u=u, post=post, gate=gate, pad=pad)


def listed():
    return [
        # one decoded token through the gated half of its 8 experts (hidden 2048, 128 experts, intermediate 768)
        _grouped("grouped T1 gate/up", 1, 8, 128, 2048, 768, True, True),
        # a decode batch of 32: two rows an expert, every expert's down matrix streamed, fp32 rows for the combine
        _grouped("grouped T32 down", 32, 8, 128, 768, 2048, False, False, y="f32"),
        # a prompt of 4096 tokens with uneven expert popularity: the gated half, rows gathered through the routing
        _grouped("grouped T4096 gate/up", 4096, 8, 128, 2048, 768, True, True, route="zipf"),
        # the same prompt's down half
        _grouped("grouped T4096 down", 4096, 8, 128, 768, 2048, False, False, y="f32", route="zipf"),
        # a verification batch of 512 over 256 large experts stored [in][out]: 16 rows an expert
        _grouped("grouped T512 large in_out", 512, 8, 256, 2048, 7168, False, False, order="in_out"),
        # odd sizes, padded rows, fp16: no dimension a multiple of a tile
        _grouped("grouped odd f16", 301, 3, 7, 1000, 1333, True, True, x="f16", y="f16", pad=24),
        # one decoded token over 4-bit experts: gated half
        _w4("w4 T1 gate/up", 1, 8, 128, 2048, 768, True, True, 128, False),
        # one decoded token through a dense 4-bit matrix the size of a shared expert's down projection
        _w4("w4 T1 dense", 1, 1, 1, 2048, 7168, False, False, 64, True, x="f16", y="f32"),
        # a decode batch of 16 over 256 large 4-bit experts with zero points
        _w4("w4 T16 large", 16, 8, 256, 7168, 2048, True, True, 32, True),
        # one token between two blocks
        _norm("norm T1", 1, 2048),
        # a prompt of 4096 tokens between two blocks, fp32 residual stream
        _norm("norm T4096", 4096, 2048),
        # a verification batch, bf16 stream of hidden 7168, a gate per channel, padded rows
        _norm("norm T512 bf16 gated", 512, 7168, x="bf16", y="bf16", gate="channel", pad=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped", "w4", "norm"))
    if op == "norm":
        H = rng.choice((_log_int(rng, 64, 8192), 4 * _log_int(rng, 16, 2048)))
        T = max(1, min(_log_int(rng, 1, 4096), (1 << 23) // H))
        return dict(op="norm", T=T, H=H, x=rng.choice((F32, BF16, F16)), y=rng.choice((F32, BF16, F16)),
                    u=rng.choice((BF16, F16)), post=rng.random() < 0.8, gate=rng.choice(("none", "channel", "token", "full")),
                    pad=rng.choice((0, 0, 8, 3)))
    while True:
        E = _log_int(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        N = _log_int(rng, 16, 7168)
        up = rng.random() < 0.5
        gather = rng.random() < 0.5
        x = rng.choice((BF16, F16))
        y = rng.choice((F32, x))
        route = rng.choice(("uniform", "zipf"))
        if op == "grouped":
            T = _log_int(rng, 1, 4096)
            K = _log_int(rng, 16, 7168)
            if E * K * N * (2 if up else 1) <= 500e6 and T * k * K * N * (2 if up else 1) <= 50e9:
                return dict(op="grouped", T=T, k=k, E=E, K=K, N=N, up=up, gather=gather, x=x, y=y,
                            order=rng.choice(("out_in", "in_out")), route=route, pad=rng.choice((0, 0, 8, 24)))
        else:
            T = _log_int(rng, 1, 64)
            group = rng.choice((32, 64, 128))
            K = group * _log_int(rng, 1, 7168 // group)
            if E * K * N * (2 if up else 1) <= 2000e6:
                return dict(op="w4", T=T, k=k, E=E, K=K, N=N, up=up, gather=gather, group=group,
                            zeros=rng.random() < 0.5, x=x, y=y, route=route, pad=rng.choice((0, 0, 8)))


# ------------------------------------------------------------------ inputs

def _pad8(n):
    return -(-n // 8) * 8


def _rows(gen, n, width, pad, dtype, scale=1.0):
    """[n, width] values in rows of at least width + pad elements."""
    full = torch.empty(n, width + pad, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
    return full[:, :width]


def _routing(case, gen):
    """Expert ids of every token, grouped: (sorted_pairs, offsets, the sizes on the host)."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.rand(T, E, device="cuda", generator=gen).clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(score))
    if case["route"] == "zipf":
        order = torch.argsort(torch.rand(E, device="cuda", generator=gen))
        log_p = -torch.log(order.float() + 1.0)
        log_p[order >= max(k, E - E // 16)] = -1e9          # some experts never asked for
        score = score + log_p
    ids = torch.topk(score, k, dim=1).indices.sort(dim=1).values.reshape(-1)
    pairs = torch.sort(ids, stable=True).indices.to(torch.int32)
    sizes = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(sizes, 0)
    return pairs, offsets, sizes.tolist()


def _quantized(gen, E, N, K, group, zeros):
    """4-bit codes, two to a byte (the even one low), scales and zero points of N(0, 0.02) weights."""
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // group, dtype=torch.float16, device="cuda")
    z = torch.empty(E, N, K // group, dtype=torch.uint8, device="cuda") if zeros else None
    for e in range(E):
        w = torch.empty(N, K // group, group, device="cuda").normal_(0.0, 0.02, generator=gen)
        if zeros:
            lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
            d = ((hi - lo) / 15).half().float()
            zp = (-lo / d).round().clamp(0, 15)
            z[e] = zp[..., 0].to(torch.uint8)
        else:
            d = (w.abs().amax(2, keepdim=True) / 7).half().float()
            zp = 8.0
        c = (w / d + zp).round().clamp(0, 15).to(torch.uint8).view(N, K)
        q[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        s[e] = d[..., 0].half()
    return q, s, z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1 + seed)
    s = dict(case=case)
    if case["op"] == "norm":
        T, H, pad = case["T"], case["H"], case["pad"]
        s["x"] = _rows(gen, T, H, pad, _DT[case["x"]], 2.0)
        s["y"] = _rows(gen, T, H, pad, _DT[case["y"]], 0.5)
        one = lambda: 1.0 + torch.empty(H, device="cuda").normal_(0.0, 0.1, generator=gen)  # noqa: E731
        s["gamma_post"] = one() if case["post"] else None
        s["gamma_pre"] = one()
        shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[case["gate"]]
        s["gate"] = torch.rand(shape, device="cuda", generator=gen) if shape else None
        s["x_out"] = torch.empty(T, H + pad, dtype=_DT[case["x"]], device="cuda")[:, :H]
        s["u"] = torch.empty(T, H, dtype=_DT[case["u"]], device="cuda")
        s["eps"], s["res_scale"], s["scale"] = 1e-6, 0.5, 1.25
        if own:
            import quantized_routed_expert_sigmoid_gb300 as moe
            s["op"] = moe.NormResidual(H, gamma_post=s["gamma_post"], gamma_pre=s["gamma_pre"], eps=s["eps"],
                                       res_scale=s["res_scale"], scale=s["scale"])
        return s
    T, k, E, K, N, up = (case[n] for n in ("T", "k", "E", "K", "N", "up"))
    dt = _DT[case["x"]]
    s["pairs"], s["offsets"], s["sizes"] = _routing(case, gen)
    rows = T if case["gather"] else T * k
    width = _pad8(K)
    s["x"] = _rows(gen, rows, width, case["pad"], dt)[:, :K]
    s["out"] = torch.empty(T * k, N, dtype=_DT[case["y"]], device="cuda")
    if case["op"] == "grouped":
        a, b = (N, K) if case["order"] == "out_in" else (K, N)
        make = lambda: torch.empty(E, a, _pad8(b), dtype=dt, device="cuda").normal_(0.0, 0.02, generator=gen)[:, :, :b]  # noqa: E731
        s["w"] = make()
        s["w_up"] = make() if up else None
    else:
        s["w"] = _quantized(gen, E, N, K, case["group"], case["zeros"])
        s["w_up"] = _quantized(gen, E, N, K, case["group"], case["zeros"]) if up else None
    if own:
        import quantized_routed_expert_sigmoid_gb300 as moe
        if case["op"] == "grouped":
            s["op"] = moe.GroupedExperts(s["w"], s["w_up"], order=case["order"], y_dtype=_DT[case["y"]])
        else:
            s["op"] = moe.W4Experts(*s["w"], up=s["w_up"], group=case["group"], x_dtype=dt, y_dtype=_DT[case["y"]])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return _plain_norm(s) if case["op"] == "norm" else _plain_products(s)
    if case["op"] == "norm":
        s["op"](s["x"], s["y"], gate=s["gate"], x_out=s["x_out"], u=s["u"])
        return [s["x_out"], s["u"]]
    return s["op"](s["x"], s["offsets"], s["pairs"] if case["gather"] else None, k=case["k"], out=s["out"])


def _plain_norm(s):
    case, n = s["case"], s["y"].float()
    if case["post"]:
        n = n * (1.0 / torch.sqrt((n * n).mean(1, keepdim=True) + s["eps"])) * s["gamma_post"]
    if s["gate"] is not None:
        n = n * s["gate"]
    r = s["res_scale"] * s["x"].float() + s["scale"] * n
    u = r * (1.0 / torch.sqrt((r * r).mean(1, keepdim=True) + s["eps"])) * s["gamma_pre"]
    return [r.to(_DT[case["x"]]), u.to(_DT[case["u"]])]


def _plain_weight(case, w, e):
    """Expert e's matrix in fp32, [N, K]."""
    if case["op"] == "grouped":
        m = w[e].float()
        return m if case["order"] == "out_in" else m.t()
    q, scale, zero = (None if t is None else t[e] for t in w)
    c = torch.stack((q & 15, q >> 4), dim=2).float().view(case["N"], -1, case["group"])
    z = 8.0 if zero is None else zero.float().unsqueeze(2)
    return ((c - z) * scale.float().unsqueeze(2)).view(case["N"], case["K"])


def _plain_products(s):
    case, out, at = s["case"], [], 0
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        rows = s["x"][torch.div(s["pairs"][at:at + n], case["k"], rounding_mode="floor")] if case["gather"] else s["x"][at:at + n]
        rows = rows.float()
        y = rows @ _plain_weight(case, s["w"], e).t()
        if case["up"]:
            y = y / (1.0 + torch.exp(-y)) * (rows @ _plain_weight(case, s["w_up"], e).t())
        out.append(y)
        at += n
    return torch.cat(out).to(_DT[case["y"]])


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, v = s["x"].double(), s["y"].double()
        if case["post"]:
            v = v / (v.pow(2).sum(1, keepdim=True) / case["H"] + s["eps"]).sqrt() * s["gamma_post"].double()
        g = 1.0 if s["gate"] is None else s["gate"].double()
        r = x * s["res_scale"] + g * v * s["scale"]
        return [r, r / (r.pow(2).sum(1, keepdim=True) / case["H"] + s["eps"]).sqrt() * s["gamma_pre"].double()]
    P, N = case["T"] * case["k"], case["N"]
    y = torch.zeros(P, N, dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    src = (s["pairs"].long() // case["k"]) if case["gather"] else torch.arange(P, device="cuda")

    def product(w, e, v):
        if case["op"] == "grouped":
            eq = "pc,nc->pn" if case["order"] == "out_in" else "pc,cn->pn"
            return torch.einsum(eq, v, w[e].double())
        q, scale, zero = w
        byte = q[e].to(torch.int64)
        code = torch.empty(N, case["K"], dtype=torch.float64, device="cuda")
        code[:, 0::2] = (byte % 16).double()
        code[:, 1::2] = (byte // 16).double()
        per = lambda t: t.double().repeat_interleave(case["group"], dim=1)  # noqa: E731
        code -= 8.0 if zero is None else per(zero[e])
        return torch.einsum("pc,nc->pn", v, per(scale[e]) * code)

    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            v = s["x"].double()[src[off[e]:off[e + 1]]] if P < 4096 else s["x"][src[off[e]:off[e + 1]]].double()
            g = product(s["w"], e, v)
            y[off[e]:off[e + 1]] = g / (1 + (-g).exp()) * product(s["w_up"], e, v) if case["up"] else g
    return y


def work(case):
    size = {BF16: 2, F16: 2, F32: 4}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        gate = {"none": 0, "channel": H, "token": T, "full": T * H}[case["gate"]]
        return {"bytes": T * H * (2 * size[case["x"]] + size[case["y"]] + size[case["u"]]) + 4 * (2 * H + gate),
                "flops": 10 * T * H}
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    if case["route"] == "zipf":
        asked = max(k, E - E // 16)
        share = [1.0 / (r + 1) for r in range(asked)]
        tot = sum(share)
        active = sum(1.0 - (1.0 - min(1.0, k * p / tot)) ** T for p in share)
    else:
        active = E * (1.0 - (1.0 - k / E) ** T)          # experts that some token is expected to ask for
    mats = 2 if case["up"] else 1
    per = 2.0 if case["op"] == "grouped" else 0.5 + (3.0 if case["zeros"] else 2.0) / case["group"]
    rows = T if case["gather"] else T * k
    return {"bytes": active * mats * N * K * per + rows * K * 2 + T * k * N * size[case["y"]]
            + 4 * (E + 1) + (4 * T * k if case["gather"] else 0), "flops": 2.0 * mats * T * k * N * K}
