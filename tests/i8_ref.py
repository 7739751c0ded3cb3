"""Plain forms of the products in 8-bit integers in 64 bits (CPU), with elementwise bounds.

Codes and whole-number sums are exact and compared for equality.  A block's h passes through its
codes: an h off by the fp32 error of its computation may round to another 16-bit number, and that
to another code, so the bound takes for each element of h the lowest and highest value that its
code may stand for (mostly one and the same).
"""
import torch

from tests import dense_ref as R

F32 = R.F32


def quant(x):
    """(codes, scales) by the definition; x [rows, n] of 16 bits.  A quotient next to a border is
    at least 2^-25 from it or on it (a multiple of half the scale's last place over the scale), which
    64 bits tell apart."""
    v = x.detach().cpu().double()
    fin = torch.isfinite(v).all(1)
    top = torch.where(fin, v.abs().amax(1), torch.zeros((), dtype=torch.float64))
    s = (top / 127).float()
    q = torch.round(torch.where(fin[:, None], v, 0.0) / torch.where(s > 0, s, 1.0).double()[:, None])
    return q.to(torch.int8), torch.where(fin, s, torch.nan)


def product(q, s, codes, scales):
    """Pair (value, bound) of ((float)sum * channel) * token: three roundings of half a step."""
    acc = q.cpu().double() @ codes.cpu().double().t()
    v = acc * scales.cpu().double()[None, :] * s.cpu().double()[:, None]
    return v, 3.1 * 2.0 ** -24 * v.abs() + R.TINY[torch.float32]


def nearest(v, dt):
    return v.to(dt).double()


def h_values(h, dt):
    """Codes, scales, and (value, lowest, highest) that the quantised h may stand for; h a pair."""
    v, e = h
    lo, hi = nearest(v - e, dt), nearest(v + e, dt)
    top_lo = torch.maximum(torch.where(lo > 0, lo, 0.0), torch.where(hi < 0, -hi, 0.0)).amax(1)
    top_hi = torch.maximum(lo.abs(), hi.abs()).amax(1)
    s_lo, s_hi = (top_lo / 127).float().double()[:, None], (top_hi / 127).float().double()[:, None]
    q, s = quant(nearest(v, dt).to(dt))
    val = q.double() * s.double()[:, None]

    def code(x, sc):
        return torch.round(x / torch.where(sc > 0, sc, 1.0)).clamp(-127, 127)

    cands = [code(x, sc) * sc2 for x in (lo, hi) for sc in (s_lo, s_hi) for sc2 in (s_lo, s_hi)]
    cands.append(val)
    return q, s, val, torch.stack(cands).amin(0), torch.stack(cands).amax(0)


def ffn(x, gate, up, down, kind, dt, residual=None, y_dt=None):
    """gate, up, down: (codes, scales).  Pair for y."""
    q, s = quant(x)
    a, u = product(q, s, *gate), product(q, s, *up)
    h = R.mul(R.act(a, kind)[0], u)
    q, s, val, lo, hi = h_values(h, dt)
    w = down[0].cpu().double() * down[1].cpu().double()[:, None]
    # by whole-number sums: those that are 0 leave nothing, a sum of rounded products would leave 2^-53 of its terms
    y = product(q, s, *down)[0]
    off = torch.maximum(hi - val, val - lo) @ w.abs().t()
    y = y, off + 3.1 * 2.0 ** -24 * (y.abs() + off) + R.TINY[torch.float32]
    if residual is not None:
        y = R.add(y, residual)
    return R.rounded(y, y_dt or dt)
