"""Plain form of the routed layer for a few tokens in 64 bits (CPU), with elementwise bounds, given the
routed experts and their gates."""
import torch

from tests import dense_ref as R
from tests import i8_ref as I8

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def record_bytes(d, f, fmt):
    return {"bf16": 6 * d * f, "mxfp4": 3 * d * f // 2 + 3 * d * f // 32, "i8": 3 * d * f + 4 * (2 * f + d)}[fmt]


def records(g, n, d, f, fmt):
    """n records of uint8 (CPU)."""
    S = record_bytes(d, f, fmt)
    if fmt == "bf16":
        return (torch.randn(n, S // 2, generator=g) * d ** -0.5).to(torch.bfloat16).view(torch.uint8)
    r = torch.randint(0, 256, (n, S), generator=g, dtype=torch.uint8)
    if fmt == "mxfp4":
        r[:, 3 * d * f // 2:] = torch.randint(119, 124, (n, 3 * d * f // 32), generator=g).to(torch.uint8)
    else:
        s = (torch.rand(n, 2 * f + d, generator=g) + 0.5) * (d ** -0.5 / 73.9)
        r[:, 3 * d * f:] = s.view(torch.uint8).reshape(n, -1)
    return r


def split(rec, d, f, fmt):
    """Three matrices: fp64 values, or (codes, scales)."""
    n = d * f
    if fmt == "bf16":
        w = rec.view(torch.bfloat16).double()
        return w[:n].reshape(f, d), w[n:2 * n].reshape(f, d), w[2 * n:].reshape(d, f)
    if fmt == "mxfp4":
        out = []
        for i, r in enumerate((f, f, d)):
            c = rec[i * n // 2:(i + 1) * n // 2].long()
            v = E2M1[torch.stack((c & 15, c >> 4), -1).reshape(-1, 32)]
            s = rec[3 * n // 2 + i * n // 32:3 * n // 2 + (i + 1) * n // 32].double()
            out.append((v * torch.exp2(s - 127)[:, None]).reshape(r, -1))
        return tuple(out)
    c, s = rec[:3 * n].view(torch.int8), rec[3 * n:].clone().view(torch.float32)
    return (c[:n].reshape(f, d), s[:f]), (c[n:2 * n].reshape(f, d), s[f:2 * f]), (c[2 * n:].reshape(d, f), s[2 * f:])


def expert(x, rec, d, f, fmt):
    """Pair for the expert's output of rows x (bf16)."""
    w = split(rec, d, f, fmt)
    if fmt == "i8":
        return I8.ffn(x, *w, "silu", torch.bfloat16, None, torch.float32)
    z = [(m, torch.zeros_like(m)) for m in w]
    xp = R.exactly(x)
    h = R.mul(R.act(R.mm(xp, R.t_(z[0])), "silu")[0], R.mm(xp, R.t_(z[1])))
    return R.mm(h, R.t_(z[2]))


def layer(x, recs, slots, idx, gates, d, f, fmt, y_dt, residual=None):
    """slots: expert -> record or None (left out).  idx, gates as the layer gave them."""
    T, k = idx.shape
    y = torch.zeros(T, d, dtype=torch.float64)
    e = torch.zeros_like(y)
    top = torch.zeros_like(y)
    for ex in idx.unique().tolist():
        s = slots.get(ex) if ex >= 0 else None
        if s is None:
            continue
        ts, js = (idx == ex).nonzero(as_tuple=True)
        v, b = expert(x[ts], recs[s], d, f, fmt)
        g = gates[ts, js].double()[:, None]
        y[ts] += g * v
        e[ts] += g * b
        top[ts] += g * (v.abs() + b)
    e += (k + 1) * R.F32 * top
    out = y, e
    if residual is not None:
        out = R.add(out, R.exactly(residual))
    return R.rounded(out, y_dt)
