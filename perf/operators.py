"""The dense operators beside the routed experts, as cases to measure: their plain forms in torch
and the library's calls (`own`).

  ffn       gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T (+ residual), also saving
            its pre-activations (16 bits or MX8) for a backward pass
  ffn_bwd   its backward pass, from saved pre-activations (16 bits or MX8) or recomputing them,
            x in 16 bits or MX8
  act8      an activation kept in 8 bits (MX8: E4M3 codes, one power-of-two scale per 32) and
            brought back
  w4        products with 4-bit weights, (code - zero) * scale per group along k
  w4_ffn    the gated block on such weights
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # one token through the shared expert of the 43-layer stack
        dict(name="ffn-t1-d4096-f2048", op="ffn", T=1, d=4096, f=2048, t="bf16", act="silu", save="none", res=False),
        # a ragged decode batch at the 40-layer stack's sizes, added to the residual stream
        dict(name="ffn-t13-d2048-f768-res", op="ffn", T=13, d=2048, f=768, t="fp16", act="silu", save="none", res=True),
        # the 8192-token prefill chunk
        dict(name="ffn-t8192-d4096-f2048", op="ffn", T=8192, d=4096, f=2048, t="bf16", act="silu", save="none", res=False),
        # a training step's forward of a wide dense layer, ragged rows, checkpoint in 8 bits
        dict(name="ffn-t2053-d4096-f11008-mx8", op="ffn", T=2053, d=4096, f=11008, t="bf16", act="gelu", save="mx8",
             res=False),
        # the backward pass of the 8192-token chunk
        dict(name="bwd-t8192-d4096-f2048", op="ffn_bwd", T=8192, d=4096, f=2048, t="bf16", act="silu", save="16",
             x8=False),
        # a short ragged step's backward pass, every activation from 8 bits
        dict(name="bwd-t1021-d2048-f5632-mx8", op="ffn_bwd", T=1021, d=2048, f=5632, t="fp16", act="silu", save="mx8",
             x8=True),
        # a chunk's activations kept and brought back; a small ragged one
        dict(name="act8-8192x4096", op="act8", T=8192, d=4096, t="bf16"),
        dict(name="act8-257x2048", op="act8", T=257, d=2048, t="fp16"),
        # one token through a square projection; a small batch through a long one with zero points
        dict(name="w4-t1-k4096-n4096-g128", op="w4", T=1, K=4096, N=4096, G=128, zero=False, t="bf16", y="fp32",
             res=False),
        dict(name="w4-t5-k11008-n4096-g64", op="w4", T=5, K=11008, N=4096, G=64, zero=True, t="fp16", y="fp16",
             res=True),
        # one token, and a decode batch of 16, through 4-bit gated blocks
        dict(name="w4ffn-t1-d4096-f11008-g128", op="w4_ffn", T=1, d=4096, f=11008, G=128, zero=False, t="bf16",
             act="silu", res=False),
        dict(name="w4ffn-t16-d4096-f2048-g32", op="w4_ffn", T=16, d=4096, f=2048, G=32, zero=True, t="bf16",
             act="silu", res=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    t = rng.choice(("bf16", "fp16"))
    act = rng.choice(("silu", "silu", "gelu"))
    op = rng.choice(("ffn", "ffn", "ffn_bwd", "ffn_bwd", "act8", "w4", "w4", "w4_ffn"))
    if op in ("ffn", "ffn_bwd"):
        save = rng.choice(("none", "16", "mx8"))
        x8 = op == "ffn_bwd" and rng.random() < 0.5
        step = 32 if save == "mx8" or x8 else 8
        d, f = _log(rng, 256, 4096, step), _log(rng, 256, 8192, step)
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 2048 // (d * f))))
        if op == "ffn":
            return dict(op=op, T=T, d=d, f=f, t=t, act=act, save=save, res=rng.random() < 0.5)
        return dict(op=op, T=T, d=d, f=f, t=t, act=act, save=save, x8=x8)
    if op == "act8":
        return dict(op=op, T=_log(rng, 1, 8192), d=_log(rng, 32, 4096, 32), t=t)
    G = rng.choice((32, 64, 128))
    zero, res, T = rng.random() < 0.5, rng.random() < 0.5, _log(rng, 1, 64)
    if op == "w4":
        return dict(op=op, T=T, K=_log(rng, 2 * G, 11008, G), N=_log(rng, 17, 11008), G=G, zero=zero, t=t,
                    y=rng.choice((t, "fp32")), res=res)
    return dict(op=op, T=T, d=_log(rng, 2 * G, 4096, G), f=_log(rng, 2 * G, 11008, G), G=G, zero=zero, t=t, act=act,
                res=res)


# ---- inputs ----------------------------------------------------------------------

def _mx8_make(g, T, n, std):
    """A tensor of N(0, std) values in MX8: codes and scales of no special rule (any code but NaN
    that such values take, under one scale a block)."""
    v = torch.randn(T, n // 32, 32, generator=g, device="cuda") * std
    top = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448))
    codes = (v / torch.exp2(e)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(T, n), (e + 127).to(torch.uint8).reshape(T, n // 32)


def _w4_make(g, N, K, G, zero, t):
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(N, K // G, generator=g, device="cuda") * 0.006 + 0.001).to(t)
    zeros = torch.randint(4, 12, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    return dict(codes=codes, scales=scales, zeros=zeros, N=N, K=K, G=G)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[case["t"]]

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)

    s = dict(case=case)
    op, T = case["op"], case["T"]
    if op in ("ffn", "ffn_bwd"):
        d, f = case["d"], case["f"]
        s |= dict(wg=rnd(f, d, std=0.02), wu=rnd(f, d, std=0.02), wd=rnd(d, f, std=0.02))
        if op == "ffn":
            s |= dict(x=rnd(T, d), res=rnd(T, d) if case["res"] else None)
        else:
            spread = 0.02 * math.sqrt(d)  # of x W^T
            s["dy"] = rnd(T, d, std=0.1)
            s["x"] = _mx8_make(g, T, d, 1.0) if case["x8"] else rnd(T, d)
            if case["save"] == "16":
                s["saved"] = rnd(2, T, f, std=spread)
            elif case["save"] == "mx8":
                a, u = _mx8_make(g, T, f, spread), _mx8_make(g, T, f, spread)
                # one buffer: codes of a and of u, then their scales
                s["saved"] = torch.cat([a[0].flatten(), u[0].flatten(), a[1].flatten(), u[1].flatten()])
        # kept between steps, as a training loop does
        s["ws"] = torch.empty(5 * T * f * 2 + T * d * 2 + (160 << 20), dtype=torch.uint8, device="cuda")
    elif op == "act8":
        s["x"] = rnd(T, case["d"])
    else:
        K = case["K"] if op == "w4" else case["d"]
        s["x"] = rnd(T, K)
        if op == "w4":
            s["w"] = _w4_make(g, case["N"], K, case["G"], case["zero"], t)
            y, n = DT[case["y"]], case["N"]
        else:
            f = case["f"]
            s |= dict(wg=_w4_make(g, f, K, case["G"], case["zero"], t), wu=_w4_make(g, f, K, case["G"], case["zero"], t),
                      wd=_w4_make(g, K, f, case["G"], case["zero"], t))
            y, n = t, K
            s["ws"] = torch.empty(T * f * 4 + (1 << 20), dtype=torch.uint8, device="cuda")
        s["res"] = torch.randn(T, n, generator=g, device="cuda").to(y) if case["res"] else None
    return s


# ---- plain forms, in 32 bits -----------------------------------------------------

def _act(a, act):
    """(act(a), act'(a))"""
    if act == "silu":
        s = 1 / (1 + torch.exp(-a))
        return a * s, s * (1 + a * (1 - s))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1 + th), 0.5 * (1 + th) + 0.5 * a * (1 - th * th) * c * (1 + 3 * 0.044715 * a * a)


def _pow2(k):
    """2^k exactly, in 64 bits (exp2 and ldexp may be an ulp off, which a border between codes sees)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _mx8_values(codes, scales, rows, n):
    """fp32 values of MX8 codes."""
    c = codes.reshape(rows, n // 32, 32).to(torch.int32)
    man, ex = c & 7, (c >> 3) & 15
    v = torch.where(ex > 0, (8 + man) * _pow2(ex - 10), man * 2.0 ** -9)
    v = torch.where(c > 127, -v, v) * _pow2(scales.reshape(rows, n // 32, 1).to(torch.int32) - 127)
    return v.reshape(rows, n).float()


def _mx8_round(v):
    """fp32 values rounded to MX8 (the values the codes stand for)."""
    b = v.reshape(v.shape[0], -1, 32).double()
    m, p = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.clamp(torch.where(m <= 0.875, p - 9, p - 8), min=-127)
    q = b * _pow2(-e)
    step = _pow2(torch.clamp(torch.frexp(q.abs())[1] - 1, min=-6) - 3)
    return (torch.round(q / step) * step * _pow2(e)).reshape(v.shape).float()


def _w4_values(w):
    """fp32 weights [N, K]."""
    c = torch.stack((w["codes"] & 15, w["codes"] >> 4), -1).reshape(w["N"], -1, w["G"]).float()
    z = 8.0 if w["zeros"] is None else w["zeros"].unsqueeze(-1).float()
    return ((c - z) * w["scales"].unsqueeze(-1).float()).reshape(w["N"], w["K"])


def _plain(s):
    c = s["case"]
    op, t = c["op"], DT[c["t"]]
    if op == "act8":
        return _mx8_round(s["x"].float()).to(t)
    if op == "w4":
        y = s["x"].float() @ _w4_values(s["w"]).t()
        return (y if s["res"] is None else y + s["res"].float()).to(DT[c["y"]])
    if op == "w4_ffn":
        x = s["x"].float()
        h = _act(x @ _w4_values(s["wg"]).t(), c["act"])[0] * (x @ _w4_values(s["wu"]).t())
        y = h @ _w4_values(s["wd"]).t()
        return (y if s["res"] is None else y + s["res"].float()).to(t)
    T, d, f = c["T"], c["d"], c["f"]
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    if op == "ffn":
        x = s["x"].float()
        a, u = x @ wg.t(), x @ wu.t()
        y = (_act(a, c["act"])[0] * u) @ wd.t()
        y = (y if s["res"] is None else y + s["res"].float()).to(t)
        if c["save"] == "16":
            return dict(y=y, a=a.to(t), u=u.to(t))
        if c["save"] == "mx8":
            return dict(y=y, a=_mx8_round(a).to(t), u=_mx8_round(u).to(t))
        return dict(y=y)
    x = _mx8_values(*s["x"], T, d) if c["x8"] else s["x"].float()
    dy = s["dy"].float()
    if c["save"] == "16":
        a, u = s["saved"].float()
    elif c["save"] == "mx8":
        v = s["saved"]
        a, u = _mx8_values(v[:2 * T * f], v[2 * T * f:], 2 * T, f).reshape(2, T, f)
    else:
        a, u = x @ wg.t(), x @ wu.t()
    act, slope = _act(a, c["act"])
    dh = dy @ wd
    da, du = dh * u * slope, dh * act
    return dict(dx=(da @ wg + du @ wu).to(t), dwg=(da.t() @ x).to(t), dwu=(du.t() @ x).to(t),
                dwd=(dy.t() @ (act * u)).to(t))


# ---- the library's calls ---------------------------------------------------------

def _own(s):
    from moe_expert_offload_amd import ft
    c = s["case"]
    op, T, t = c["op"], c["T"], DT[c["t"]]
    dt = {"bf16": ft.FT_T_BF16, "fp16": ft.FT_T_FP16, "fp32": ft.FT_T_FP32}
    if op == "act8":
        n = c["d"]
        codes = torch.empty((T, n), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, n // 32), dtype=torch.uint8, device="cuda")
        ft.ft_act8_pack(s["x"], n, T, n, dt[c["t"]], codes, scales)
        out = torch.empty((T, n), dtype=t, device="cuda")
        ft.ft_act8_unpack(codes, scales, T, n, dt[c["t"]], out, n)
        return out
    if op in ("w4", "w4_ffn"):
        def matrix(w):
            return ft.make_w4_matrix(w["codes"], w["scales"], w["zeros"], w["N"], w["K"], w["G"])
        x, res = s["x"], s["res"]
        if op == "w4":
            n = c["N"]
            y = torch.empty((T, n), dtype=DT[c["y"]], device="cuda")
            ft.ft_w4_gemv(x, c["K"], T, dt[c["t"]], matrix(s["w"]), res, n, y, n, dt[c["y"]])
            return y
        d = c["d"]
        y = torch.empty((T, d), dtype=t, device="cuda")
        act = ft.FT_ACT_SILU if c["act"] == "silu" else ft.FT_ACT_GELU_TANH
        ft.ft_w4_gated_ffn(x, d, T, dt[c["t"]], act, matrix(s["wg"]), matrix(s["wu"]), matrix(s["wd"]), res, d, y, d,
                           dt[c["t"]], s["ws"], s["ws"].numel())
        return y
    d, f = c["d"], c["f"]
    act = ft.FT_ACT_SILU if c["act"] == "silu" else ft.FT_ACT_GELU_TANH
    fmt = {"none": ft.FT_SAVE_NONE, "16": ft.FT_SAVE_16, "mx8": ft.FT_SAVE_MX8}[c["save"]]
    ws = s["ws"]
    if op == "ffn":
        y = torch.empty((T, d), dtype=t, device="cuda")
        if c["save"] == "16":
            saved = torch.empty((2, T, f), dtype=t, device="cuda")
        elif c["save"] == "mx8":
            saved = torch.empty(2 * T * f + 2 * T * (f // 32), dtype=torch.uint8, device="cuda")
        else:
            saved = None
        ft.ft_gated_ffn(s["x"], d, T, d, f, dt[c["t"]], act, s["wg"], s["wu"], s["wd"], s["res"], d, y, d, dt[c["t"]],
                        saved, fmt, ws, ws.numel())
        if c["save"] == "16":
            return dict(y=y, a=saved[0], u=saved[1])
        if c["save"] == "mx8":
            values = torch.empty((2, T, f), dtype=t, device="cuda")
            ft.ft_act8_unpack(saved, saved[2 * T * f:], 2 * T, f, dt[c["t"]], values, f)
            return dict(y=y, a=values[0], u=values[1])
        return dict(y=y)
    x, xs = s["x"] if c["x8"] else (s["x"], None)
    dx = torch.empty((T, d), dtype=t, device="cuda")
    dwg, dwu = torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
    dwd = torch.empty_like(s["wd"])
    ft.ft_gated_ffn_bwd(x, d, xs, T, d, f, dt[c["t"]], act, s["wg"], s["wu"], s["wd"], s.get("saved"), fmt, s["dy"], d,
                        dx, d, dwg, dwu, dwd, ws, ws.numel())
    return dict(dx=dx, dwg=dwg, dwu=dwu, dwd=dwd)


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_act(a, act):
    if act == "silu":
        return a * torch.sigmoid(a)
    return a / 2 * (1 + torch.tanh((a + 0.044715 * a ** 3) * (2 / math.pi) ** 0.5))


def _exact_pow2(k):
    table = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device="cuda")
    return table[k.long() + 160]


def _exact_mx8_decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * _exact_pow2(scales.long() - 127).repeat_interleave(32, dim=1)


def _exact_mx8_round(v):
    """The nearest of the E4M3 points under each block's scale, ties to the even code."""
    points = torch.arange(127, device=v.device)
    ex, man = points // 8, points % 8
    points = torch.where(ex > 0, (1 + man.double() / 8) * _exact_pow2(ex - 7), man.double() * 2.0 ** -9)
    b = v.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    bounds = 448 * _exact_pow2(torch.arange(-127, 140))  # the least of these that holds the block's largest
    e = torch.searchsorted(bounds, top) - 127
    q = b.abs() / _exact_pow2(e)
    hi = torch.searchsorted(points, q.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = points[hi] - q, q - points[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(b) * points[code] * _exact_pow2(e)).reshape(v.shape)


def _exact_w4(w):
    lo, hi = w["codes"].double() % 16, torch.div(w["codes"], 16, rounding_mode="floor").double()
    q = torch.empty(w["N"], w["K"], dtype=torch.float64, device="cuda")
    q[:, 0::2], q[:, 1::2] = lo, hi
    z = torch.full_like(w["scales"], 8.0) if w["zeros"] is None else w["zeros"]
    return (q - z.double().repeat_interleave(w["G"], 1)) * w["scales"].double().repeat_interleave(w["G"], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        return _exact_mx8_round(s["x"].double())
    if op in ("w4", "w4_ffn"):
        x = s["x"].double()
        if op == "w4":
            y = torch.matmul(_exact_w4(s["w"]), x.t()).t()
        else:
            a, u = (torch.matmul(_exact_w4(s[k]), x.t()) for k in ("wg", "wu"))
            y = torch.matmul(_exact_w4(s["wd"]), _exact_act(a, case["act"]) * u).t()
        return y.contiguous() if s["res"] is None else y + s["res"].double()
    wg, wu, wd = (s[k].double() for k in ("wg", "wu", "wd"))
    T, d, f = case["T"], case["d"], case["f"]
    if op == "ffn":
        x = s["x"].double()
        a, u = torch.matmul(wg, x.t()).t(), torch.matmul(wu, x.t()).t()
        y = torch.matmul(wd, (_exact_act(a, case["act"]) * u).t()).t()
        out = dict(y=y.contiguous() if s["res"] is None else y + s["res"].double())
        if case["save"] != "none":
            keep = _exact_mx8_round if case["save"] == "mx8" else (lambda v: v)
            out |= dict(a=keep(a.contiguous()), u=keep(u.contiguous()))
        return out
    x = _exact_mx8_decode(*s["x"]) if case["x8"] else s["x"].double()
    for v in (x, wg, wu, wd):
        v.requires_grad_(True)
    a, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    if case["save"] == "16":  # the block's own values stand in the product, its slopes in the gradients
        ka, ku = s["saved"].double()
    elif case["save"] == "mx8":
        v = s["saved"]
        n = 2 * T * f
        ka, ku = _exact_mx8_decode(v[:n].reshape(2 * T, f), v[n:].reshape(2 * T, f // 32)).reshape(2, T, f)
    else:
        ka, ku = a.detach(), u.detach()
    y = torch.matmul(_exact_act(a + (ka - a.detach()), case["act"]) * (u + (ku - u.detach())), wd.t())
    dx, dwg, dwu, dwd = torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].double())
    return dict(dx=dx, dwg=dwg, dwu=dwu, dwd=dwd)


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "act8":
        n = T * case["d"]
        return {"bytes": 2 * n + 2 * (n + n // 32) + 2 * n, "flops": 4 * n}
    if op in ("w4", "w4_ffn"):
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        per = 0.5 + (2 + (1 if case["zero"] else 0)) / case["G"]
        K = case["K"] if op == "w4" else case["d"]
        out = case["N"] if op == "w4" else case["d"]
        weights = K * case["N"] if op == "w4" else 3 * K * case["f"]
        y = size[case["y"] if op == "w4" else case["t"]]
        return {"bytes": int(weights * per) + 2 * T * K + T * out * y * (2 if case["res"] else 1),
                "flops": 2 * T * weights}
    d, f = case["d"], case["f"]
    kept = {"none": 0, "16": 2 * T * f * 2, "mx8": 2 * T * (f + f // 32)}[case["save"]]
    if op == "ffn":
        return {"bytes": 3 * d * f * 2 + T * d * (6 if case["res"] else 4) + kept, "flops": 6 * T * d * f}
    x = T * (d + d // 32) if case["x8"] else T * d * 2
    return {"bytes": 2 * 3 * d * f * 2 + x + 2 * T * d * 2 + kept,
            "flops": (16 if case["save"] == "none" else 12) * T * d * f}
