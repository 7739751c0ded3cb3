"""Plain forms of the dense operators in 64 bits (CPU), with elementwise error bounds.

A quantity is a pair (value, bound): the exact value for the inputs, and how far a computation
in fp32 with the documented roundings to 16 bits may be from it.
  - a sum of K products in fp32 is off by at most K steps of its terms' magnitudes: each
    addition rounds by at most 2^-23 of the partial sum (2^-24 to nearest; the matrix cores'
    inner additions may truncate), and partial sums stay below the sum of magnitudes;
  - rounding to 16 bits is off by half a step, finfo.eps / 2 of the value, or half the smallest
    subnormal;
  - exp and the reciprocal of the activations are within a few ulp, and exp's argument z is
    itself rounded, which makes |z| 2^-24 relative more.
"""
import math

import torch

F32 = 2.0 ** -23
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def exactly(t, on="cpu"):
    """on: where the 64-bit work is done (large cases: the GPU's own 64-bit products)."""
    v = t.detach().to(on).double()
    return v, torch.zeros_like(v)


def mm(a, b):
    """a [m, k] times b [k, n]."""
    (av, ae), (bv, be) = a, b
    aa, ba = av.abs() + ae, bv.abs() + be
    return av @ bv, aa @ ba - av.abs() @ bv.abs() + (av.shape[1] + 1) * F32 * (aa @ ba)


def t_(a):
    return a[0].t(), a[1].t()


def add(a, b):
    s = a[0] + b[0]
    return s, a[1] + b[1] + F32 * (s.abs() + a[1] + b[1])


def mul(a, b):
    p = a[0] * b[0]
    top = (a[0].abs() + a[1]) * (b[0].abs() + b[1])
    return p, top - p.abs() + F32 * top


def rounded(a, dt):
    u = torch.finfo(dt).eps / 2
    return a[0], a[1] + u * (a[0].abs() + a[1]) + TINY[dt]


def act(a, kind):
    """(act(a), act'(a)).  |act'| <= 1.2 and |act''| <= 1.2 for both kinds."""
    v, e = a
    if kind == "silu":
        s = torch.sigmoid(v)
        f, df = v * s, s * (1 + v * (1 - s))
        rel = (v.abs() + 16) * F32
        slope = (s * (1 - s) * (v.abs() + 1) + s)
    else:
        c = math.sqrt(2 / math.pi)
        w = c * (v + 0.044715 * v ** 3)
        s = torch.sigmoid(2 * w)
        f, df = v * s, s + v * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * v * v)
        rel = (8 * w.abs() + 16) * F32
        slope = s + v.abs() * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * v * v)
    # s is off by rel s (1 - s) and a little of s; 1 - s is a difference of values near 1
    return (f, 1.2 * e + rel * f.abs() + TINY[torch.float32]), (df, 1.2 * e + rel * (slope + v.abs() * s) + TINY[torch.float32])


def ffn(x, wg, wu, wd, kind, dt, residual=None, y_dt=None):
    """Forward: dict of pairs a, u, h, y; x, wg, wu, wd pairs."""
    a, u = mm(x, t_(wg)), mm(x, t_(wu))
    h = rounded(mul(act(a, kind)[0], u), dt)
    y = mm(h, t_(wd))
    if residual is not None:
        y = add(y, residual)
    return dict(a=a, u=u, h=h, y=rounded(y, y_dt or dt))


def ffn_bwd(x, wg, wu, wd, a, u, dy, kind, dt):
    f, df = act(a, kind)
    h = rounded(mul(f, u), dt)
    dh = mm(dy, wd)
    da, du = rounded(mul(mul(dh, u), df), dt), rounded(mul(dh, f), dt)
    dx = add(mm(da, wg), mm(du, wu))
    # one running sum over both products
    dx = dx[0], dx[1] + (wg[0].shape[0] + 1) * F32 * (da[0].abs() @ wg[0].abs() + du[0].abs() @ wu[0].abs())
    return {k: rounded(v, dt) for k, v in dict(dx=dx, dwg=mm(t_(da), x), dwu=mm(t_(du), x), dwd=mm(t_(dy), h)).items()}


def check(got, want, what=""):
    """Every element within its bound; prints the worst use of it."""
    v, e = want
    g = got.detach().to(v.device).double()
    assert g.shape == v.shape, (what, g.shape, v.shape)
    assert torch.isfinite(g).all(), what
    use = ((g - v).abs() / e).max().item() if g.numel() else 0.0
    print(f"[bound] {what}: {use:.3f} of the bound", flush=True)
    assert use <= 1.0, (what, use)


# ---- MX8 ---------------------------------------------------------------------------

def e4m3_points():
    """The 127 magnitudes of E4M3 codes 0..126."""
    return torch.tensor([(c % 8) * 2.0 ** -9 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7) for c in range(127)],
                        dtype=torch.float64)


def mx8_values(codes, scales):
    """fp64 values of codes [rows, n] under scales [rows, n / 32]; NaN codes give NaN."""
    pts = torch.cat([e4m3_points(), torch.tensor([math.nan], dtype=torch.float64)])
    c = codes.cpu().long()
    v = pts[c & 127] * torch.where(c > 127, -1.0, 1.0).double()
    e = scales.cpu().long() - 127
    table = torch.tensor([2.0 ** k for k in range(-127, 129)], dtype=torch.float64)
    return v * table[e + 127].repeat_interleave(32, dim=1)


def mx8_pack(v):
    """(codes, scales) of fp64 values [rows, n] by the definition, by search over all points."""
    rows, n = v.shape
    b = v.reshape(-1, 32)
    fin = torch.isfinite(b)
    top = torch.where(fin, b.abs(), 0.0).amax(1)
    bounds = torch.tensor([448.0 * 2.0 ** e for e in range(-127, 121)], dtype=torch.float64)
    e = torch.searchsorted(bounds, top)  # the least e + 127 with top <= 448 2^e
    e = torch.where(top == 0, torch.zeros_like(e), e)
    q = b.abs() / torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64)[e].unsqueeze(1)
    d = (torch.where(fin, q, 0.0).unsqueeze(-1) - e4m3_points()).abs()
    near = d.amin(-1, keepdim=True)
    cand = torch.arange(127).expand(d.shape)
    even = torch.where((d == near) & (cand % 2 == 0), cand, 1000).amin(-1)
    any_ = torch.where(d == near, cand, 1000).amin(-1)
    code = torch.where(even < 1000, even, any_)
    code = torch.where(fin, code, 127)
    neg = torch.signbit(b)
    return (code + 128 * neg).to(torch.uint8).reshape(rows, n), e.to(torch.uint8).reshape(rows, n // 32)


# ---- 4-bit weights ------------------------------------------------------------------

def w4_values(codes, scales, zeros, group):
    c = codes.cpu().long()
    q = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1).double()
    z = torch.full(scales.shape, 8.0, dtype=torch.float64) if zeros is None else zeros.cpu().double()
    return (q - z.repeat_interleave(group, 1)) * scales.cpu().double().repeat_interleave(group, 1)


def w4_mm(x, w, codes, scales, zeros, group):
    """x pair [T, K] times w^T with the kernel's bound: a group's sum runs over (16 + code) x and
    -(16 + zero) x, terms of up to 31 |x|, before the scale; the groups' sums are then added."""
    xv, xe = x
    y = xv @ w.t()
    # 2 K terms of magnitude at most 31 |x| scale, and the groups' additions
    s = scales.cpu().double().abs().repeat_interleave(group, 1)
    top = (xv.abs() + xe) @ (31 * s).t()
    # partial sums inside a group never exceed the group's own terms
    return y, xe @ w.abs().t() + (2 * group + xv.shape[1] / group + 8) * F32 * top
