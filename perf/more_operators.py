"""Operators on 8-bit integers and the whole routed layer for a few tokens, as cases to measure:
their plain forms in torch and the library's calls (`own`).

  quant   rows to 8-bit integers under one scale each: s = max|x| / 127, code = round(x / s)
  gemm    y = x w^T of such rows (given so, or quantised on the way) and 8-bit weights with a
          scale for each channel (+ residual)
  ffn     the gated block y = quant(act(x Wg^T) * (x Wu^T)) Wd^T (+ residual) on such weights
  moe     a routed layer whose experts are all on the device: router, top-k, gates, the experts
          of each token (bf16, MXFP4 or 8-bit records), their weighted sum (+ residual)
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # an 8192-token chunk's activations before an 8-bit product; a small ragged batch
        dict(name="quant-8192x4096", op="quant", T=8192, K=4096, t="bf16"),
        dict(name="quant-257x2048", op="quant", T=257, K=2048, t="fp16"),
        # one token through a square projection; a ragged decode batch through a long one
        dict(name="gemm-t1-k4096-n4096", op="gemm", T=1, K=4096, N=4096, x8=False, t="bf16", y="bf16", res=False),
        dict(name="gemm-t13-k11008-n4099-res", op="gemm", T=13, K=11008, N=4099, x8=False, t="fp16", y="fp32", res=True),
        # a ragged middle-sized batch; the 8192-token chunk, quantised before (its codes feed more than one product)
        dict(name="gemm-t1021-k2048-n5632", op="gemm", T=1021, K=2048, N=5632, x8=False, t="bf16", y="bf16", res=False),
        dict(name="gemm-t8192-k4096-n4096", op="gemm", T=8192, K=4096, N=4096, x8=True, t="bf16", y="bf16", res=False),
        # one token, and the 8192-token chunk, through gated blocks
        dict(name="ffn-t1-d4096-f11008", op="ffn", T=1, d=4096, f=11008, t="bf16", act="silu", res=False),
        dict(name="ffn-t8192-d4096-f2048-res", op="ffn", T=8192, d=4096, f=2048, t="bf16", act="silu", res=True),
        # one token through a layer of the 43-layer stack, bf16 records
        dict(name="moe-t1-d4096-f2048-e256-k6-bf16", op="moe", T=1, d=4096, f=2048, E=256, k=6, fmt="bf16", y="fp32",
             mask=False, res=False),
        # the same in MXFP4, a decode batch
        dict(name="moe-t16-d4096-f2048-e256-k6-mxfp4", op="moe", T=16, d=4096, f=2048, E=256, k=6, fmt="mxfp4", y="fp32",
             mask=False, res=True),
        # one token through a layer of the 40-layer stack, 8-bit records
        dict(name="moe-t1-d2048-f768-e128-k8-i8", op="moe", T=1, d=2048, f=768, E=128, k=8, fmt="i8", y="bf16",
             mask=False, res=False),
        # a ragged decode batch there, some experts not allowed
        dict(name="moe-t13-d2048-f768-e128-k8-i8", op="moe", T=13, d=2048, f=768, E=128, k=8, fmt="i8", y="bf16",
             mask=True, res=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(("quant", "gemm", "gemm", "ffn", "ffn", "moe", "moe", "moe"))
    t = rng.choice(("bf16", "fp16"))
    res = rng.random() < 0.5
    if op == "quant":
        return dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 16, 4096, 16), t=t)
    if op == "gemm":
        K, N = _log(rng, 128, 11008, 16), _log(rng, 17, 11008)
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 4096 // (K * N))))
        return dict(op=op, T=T, K=K, N=N, x8=rng.random() < 0.5, t=t, y=rng.choice((t, "fp32")), res=res)
    if op == "ffn":
        d, f = _log(rng, 256, 4096, 16), _log(rng, 256, 11008, 16)
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 2048 // (d * f))))
        return dict(op=op, T=T, d=d, f=f, t=t, act=rng.choice(("silu", "silu", "gelu")), res=res)
    fmt = rng.choice(("bf16", "mxfp4", "i8"))
    sd, sf = {"bf16": (8, 8), "mxfp4": (256, 128), "i8": (16, 16)}[fmt]
    case = dict(op=op, T=_log(rng, 1, 64), d=_log(rng, 256, 4096, sd), f=_log(rng, 128, 2048, sf), E=_log(rng, 8, 256),
                k=rng.randint(1, 8), fmt=fmt, y="bf16" if fmt == "i8" else rng.choice(("bf16", "fp32")),
                mask=rng.random() < 0.3, res=res)
    most = max((work(c) for c in listed() if c["op"] == "moe"), key=lambda w: w["bytes"])
    while any(work(case)[n] > most[n] for n in most):  # as many tokens as the largest listed layer's cost allows
        case["T"] -= 1
    return case


# ---- inputs ----------------------------------------------------------------------

def _i8_make(g, N, K, std):
    """8-bit weights whose values have about that standard deviation, channels of different sizes."""
    codes = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    scales = (torch.rand(N, generator=g, device="cuda") + 0.5) * (std / 73.3)
    return dict(codes=codes, scales=scales, N=N, K=K)


def _record_bytes(d, f, fmt):
    return {"bf16": 6 * d * f, "mxfp4": 3 * d * f // 2 + 3 * d * f // 32, "i8": 3 * d * f + 4 * (2 * f + d)}[fmt]


def _records(g, E, d, f, fmt):
    """E expert records, one after another."""
    S = _record_bytes(d, f, fmt)
    if fmt == "bf16":
        r = torch.empty(E, S // 2, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02, generator=g)
        return r.view(torch.uint8)
    r = torch.empty(E, S, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    if fmt == "mxfp4":  # scales of 2^-9 .. 2^-5 behind the codes
        r[:, 3 * d * f // 2:] %= 5
        r[:, 3 * d * f // 2:] += 118
    else:
        s = (torch.rand(E, 2 * f + d, generator=g, device="cuda") + 0.5) * (0.02 / 73.3)
        r[:, 3 * d * f:] = s.view(torch.uint8)
    return r


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]

    def rnd(*shape, std=1.0, t=DT[case["t"]] if "t" in case else torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)

    s = dict(case=case)
    ws = 0  # a workspace kept between calls, as a serving loop does
    if op == "quant":
        s["x"] = rnd(T, case["K"])
    elif op == "gemm":
        K, N = case["K"], case["N"]
        if case["x8"]:
            s["x"] = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
            s["xs"] = (torch.rand(T, generator=g, device="cuda") + 0.5) * 0.02
        else:
            s["x"], s["xs"] = rnd(T, K), None
        s["w"] = _i8_make(g, N, K, 0.02)
        s["res"] = rnd(T, N, t=DT[case["y"]]) if case["res"] else None
        ws = T * K + 4 * T + (160 << 20)
    elif op == "ffn":
        d, f = case["d"], case["f"]
        s |= dict(x=rnd(T, d), wg=_i8_make(g, f, d, 0.02), wu=_i8_make(g, f, d, 0.02), wd=_i8_make(g, d, f, 0.02),
                  res=rnd(T, d) if case["res"] else None)
        ws = T * d + 3 * T * f + 8 * T + (160 << 20)
    else:
        d, f, E, k = case["d"], case["f"], case["E"], case["k"]
        s |= dict(x=rnd(T, d), wr=rnd(E, d, std=d ** -0.5), records=_records(g, E, d, f, case["fmt"]))
        # about a quarter of the experts not allowed, k of them always
        s["allowed"] = None
        if case["mask"]:
            u = torch.rand(T, E, generator=g, device="cuda")
            s["allowed"] = (u <= torch.clamp(u.sort(1)[0][:, k - 1:k], min=0.75)).to(torch.uint8)
        s["res"] = rnd(T, d, t=DT[case["y"]]) if case["res"] else None
        ws = T * k * f * 4 + T * d * 4 + T * E * 4 + (1 << 20)
    if ws:
        s["ws"] = torch.empty(ws, dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms, in 32 bits -----------------------------------------------------

def _act(a, act):
    if act == "silu":
        return a / (1 + torch.exp(-a))
    return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))


def _quant(x):
    """Codes (as fp32 numbers) and scales of rows; in 64 bits, since values lie next to the borders between codes."""
    s = (x.abs().amax(-1).double() / 127).float()
    q = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1))
    return q.float(), s


def _i8_mm(q, s, codes, scales):
    """Products of whole numbers pass 2^24: their sums in 64 bits."""
    return (q.double() @ codes.double().t()).float() * scales * s.unsqueeze(-1)


def _i8_block(x, wg, wu, wd, act, t):
    """x [T, d] in its 16-bit type; (codes, scales) of each matrix."""
    q, s = _quant(x)
    h = (_act(_i8_mm(q, s, *wg), act) * _i8_mm(q, s, *wu)).to(t)  # the block keeps h in its type before the codes
    q, s = _quant(h)
    return _i8_mm(q, s, *wd)


def _mx_values(codes, scales):
    """fp32 weights of E2M1 codes [..., n / 2] under a power of two per 32."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1, 32).to(torch.int32)
    m, e = c & 1, (c >> 1) & 3
    v = torch.where(e > 0, (2 + m).float() * torch.exp2((e - 2).float()), m.float() * 0.5)
    v = torch.where(c > 7, -v, v) * torch.exp2(scales.float() - 127).unsqueeze(-1)
    return v.reshape(codes.shape[0], -1)


def _split(rec, d, f, fmt):
    """The three matrices of one record: fp32 values, or codes and scales."""
    n = d * f
    if fmt == "bf16":
        w = rec.view(torch.bfloat16)
        return [w[i * n:(i + 1) * n].reshape(r, -1).float() for i, r in enumerate((f, f, d))]
    if fmt == "mxfp4":
        sc = rec[3 * n // 2:]
        return [_mx_values(rec[i * n // 2:(i + 1) * n // 2].reshape(r, -1), sc[i * n // 32:(i + 1) * n // 32].reshape(r, -1))
                for i, r in enumerate((f, f, d))]
    codes, sc = rec[:3 * n].view(torch.int8), rec[3 * n:].view(torch.float32)
    return [(codes[:n].reshape(f, d), sc[:f]), (codes[n:2 * n].reshape(f, d), sc[f:2 * f]),
            (codes[2 * n:].reshape(d, f), sc[2 * f:])]


def _plain_moe(s):
    c = s["case"]
    T, d, f, k, fmt = c["T"], c["d"], c["f"], c["k"], c["fmt"]
    x = s["x"]
    logits = x.double() @ s["wr"].double().t()  # in 64 bits: which experts are taken hangs on their order
    if s["allowed"] is not None:
        logits = torch.where(s["allowed"] != 0, logits, torch.full_like(logits, -math.inf))
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k].float(), idx[:, :k]
    e = torch.exp(top - top[:, :1])
    gates = e / e.sum(1, keepdim=True)
    y = torch.zeros(T, d, device="cuda") if s["res"] is None else s["res"].float()
    rows = []
    for t in range(T):
        recs, acc = torch.index_select(s["records"], 0, idx[t]), y[t:t + 1]
        for j in range(k):
            w = _split(recs[j], d, f, fmt)
            if fmt == "i8":
                out = _i8_block(x[t:t + 1], *w, "silu", torch.bfloat16)
            else:
                xf = x[t:t + 1].float()
                out = (_act(xf @ w[0].t(), "silu") * (xf @ w[1].t())) @ w[2].t()
            acc = acc + gates[t, j] * out
        rows.append(acc)
    return dict(y=torch.cat(rows).to(DT[c["y"]]), idx=idx.to(torch.int32), gates=gates)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "moe":
        return _plain_moe(s)
    if op == "quant":
        q, sc = _quant(s["x"])
        return dict(codes=q.to(torch.int8), scales=sc)
    res = 0 if s["res"] is None else s["res"].float()
    if op == "gemm":
        q, sc = (s["x"].float(), s["xs"]) if c["x8"] else _quant(s["x"])
        return (_i8_mm(q, sc, s["w"]["codes"], s["w"]["scales"]) + res).to(DT[c["y"]])
    w = [(s[n]["codes"], s[n]["scales"]) for n in ("wg", "wu", "wd")]
    return (_i8_block(s["x"], *w, c["act"], DT[c["t"]]) + res).to(DT[c["t"]])


# ---- the library's calls ---------------------------------------------------------

def _own(s):
    from moe_expert_offload_amd import ft
    c = s["case"]
    op, T = c["op"], c["T"]
    dt = {"bf16": ft.FT_T_BF16, "fp16": ft.FT_T_FP16, "fp32": ft.FT_T_FP32}
    if op == "quant":
        n = c["K"]
        codes = torch.empty((T, n), dtype=torch.int8, device="cuda")
        scales = torch.empty(T, dtype=torch.float32, device="cuda")
        ft.ft_i8_quant(s["x"], n, T, n, dt[c["t"]], codes, scales)
        return dict(codes=codes, scales=scales)
    ws = s["ws"]

    def matrix(w):
        return ft.make_i8_matrix(w["codes"], w["scales"], w["N"], w["K"])

    if op == "gemm":
        K, N = c["K"], c["N"]
        y = torch.empty((T, N), dtype=DT[c["y"]], device="cuda")
        ft.ft_i8_gemm(s["x"], K, s["xs"], T, dt[c["t"]], matrix(s["w"]), s["res"], N, y, N, dt[c["y"]], ws, ws.numel())
        return y
    d = c["d"]
    if op == "ffn":
        y = torch.empty((T, d), dtype=DT[c["t"]], device="cuda")
        act = ft.FT_ACT_SILU if c["act"] == "silu" else ft.FT_ACT_GELU_TANH
        ft.ft_i8_gated_ffn(s["x"], d, T, dt[c["t"]], act, matrix(s["wg"]), matrix(s["wu"]), matrix(s["wd"]), s["res"], d,
                           y, d, dt[c["t"]], ws, ws.numel())
        return y
    k, E = c["k"], c["E"]
    fmt = {"bf16": ft.FT_W_BF16, "mxfp4": ft.FT_W_MXFP4, "i8": ft.FT_W_I8}[c["fmt"]]
    y = torch.empty((T, d), dtype=DT[c["y"]], device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), dtype=torch.float32, device="cuda")
    ft.ft_moe_layer(ft.make_shape(1, E, d, c["f"], k, fmt), s["x"], T, s["wr"], s["allowed"], s["records"], E, None,
                    s["res"], y, dt[c["y"]], idx, gates, ws, ws.numel())
    return dict(y=y, idx=idx, gates=gates)


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_act(a, act):
    if act == "silu":
        return a * torch.sigmoid(a)
    return a / 2 * (1 + torch.tanh((a + 0.044715 * a ** 3) * (2 / math.pi) ** 0.5))


def _exact_quant(x):
    """(codes, scales) in 64 bits; the scale itself is an fp32 number by definition."""
    x = x.double()
    top = torch.linalg.vector_norm(x, math.inf, dim=1)
    s = torch.div(top, 127.0).to(torch.float32).double()
    inv = x / s.clamp(min=1e-300)[:, None]
    lo = torch.floor(inv)
    up = (inv - lo > 0.5) | ((inv - lo == 0.5) & (torch.remainder(lo, 2) == 1))
    return lo + up, s


def _exact_rows(x, codes, scales):
    """Rows of 16 bits, quantised, times 8-bit weights."""
    q, s = _exact_quant(x)
    return torch.matmul(codes.double(), q.t()).t() * scales.double()[None, :] * s[:, None]


def _exact_block(x, w, act, t):
    a, u = _exact_rows(x, *w[0]), _exact_rows(x, *w[1])
    return _exact_rows((_exact_act(a, act) * u).to(t), *w[2])


def _exact_mx(codes, scales, rows):
    points = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    v = torch.empty(codes.numel() * 2, dtype=torch.float64, device="cuda")
    v[0::2], v[1::2] = points[(codes % 16).long()], points[torch.div(codes, 16, rounding_mode="floor").long()]
    pow2 = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")
    return (v.reshape(-1, 32) * pow2[scales.long()][:, None]).reshape(rows, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        q, sc = _exact_quant(s["x"])
        return dict(codes=q, scales=sc)
    res = 0.0 if s["res"] is None else s["res"].double()
    if op == "gemm":
        if case["x8"]:
            y = torch.matmul(s["w"]["codes"].double(), s["x"].double().t()).t()
            return y * s["w"]["scales"].double()[None, :] * s["xs"].double()[:, None] + res
        return _exact_rows(s["x"], s["w"]["codes"], s["w"]["scales"]) + res
    if op == "ffn":
        w = [(s[n]["codes"], s[n]["scales"]) for n in ("wg", "wu", "wd")]
        return _exact_block(s["x"], w, case["act"], DT[case["t"]]) + res
    T, d, f, k, fmt = case["T"], case["d"], case["f"], case["k"], case["fmt"]
    n = d * f
    logits = torch.matmul(s["wr"].double(), s["x"].double().t()).t().cpu()
    idx = torch.empty(T, k, dtype=torch.int64)
    for t in range(T):
        order = sorted((-logits[t, e].item(), e) for e in range(case["E"]) if s["allowed"] is None or s["allowed"][t, e])
        idx[t] = torch.tensor([e for _, e in order[:k]])
    gates = torch.softmax(torch.gather(logits, 1, idx), dim=1)
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda") + res
    for e in idx.unique().tolist():
        rec = s["records"][e]
        ts, js = (idx == e).nonzero(as_tuple=True)
        x = s["x"][ts.cuda()]
        if fmt == "i8":
            c, sc = rec[:3 * n].view(torch.int8).reshape(3, n), rec[3 * n:].view(torch.float32)
            out = _exact_block(x, [(c[0].view(f, d), sc[:f]), (c[1].view(f, d), sc[f:2 * f]), (c[2].view(d, f), sc[2 * f:])],
                               "silu", torch.bfloat16)
        else:
            if fmt == "bf16":
                wg, wu, wd = (m.double().reshape(r, -1) for m, r in zip(rec.view(torch.bfloat16).reshape(3, n), (f, f, d)))
            else:
                c, sc = rec[:3 * n // 2].reshape(3, -1), rec[3 * n // 2:].reshape(3, -1)
                wg, wu, wd = (_exact_mx(c[i], sc[i], r) for i, r in enumerate((f, f, d)))
            x = x.double()
            h = _exact_act(torch.matmul(wg, x.t()), "silu") * torch.matmul(wu, x.t())
            out = torch.matmul(wd, h).t()
        y[ts.cuda()] += gates[ts, js].cuda()[:, None] * out
    return dict(y=y, idx=idx.cuda(), gates=gates.cuda())


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "quant":
        n = T * case["K"]
        return {"bytes": 3 * n + 4 * T, "flops": 3 * n}
    if op == "gemm":
        K, N = case["K"], case["N"]
        x = T * K + 4 * T if case["x8"] else 2 * T * K
        return {"bytes": x + N * K + 4 * N + T * N * size[case["y"]] * (2 if case["res"] else 1), "flops": 2 * T * N * K}
    d, f = case["d"], case["f"]
    if op == "ffn":
        return {"bytes": 3 * d * f + 4 * (2 * f + d) + 2 * T * d * (3 if case["res"] else 2), "flops": 6 * T * d * f}
    # the distinct experts that T tokens with k of E each meet when all are equally likely
    E, k = case["E"], case["k"]
    used = E * (1 - (1 - k / E) ** T)
    io = T * d * (2 + size[case["y"]] * (2 if case["res"] else 1)) + T * k * 8 + (T * E if case["mask"] else 0)
    return {"bytes": int(2 * E * d + used * _record_bytes(d, f, case["fmt"])) + io, "flops": T * (2 * E * d + 6 * k * d * f)}
