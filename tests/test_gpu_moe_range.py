"""GPU tests of the routed layer's range with MXFP4 records: a block's sum of 32 products is made before its scale is applied,
so x and h may be as large as 6 sum |v| over a block allows, 1.7e36 for equal ones, whatever the scales."""
import pytest

from tests import dense_ref as R
from tests import moe_ref as M
from tests.gpu_helpers import torch_mod
from tests.test_gpu_moe_layer import Layer, _say

pytestmark = pytest.mark.gpu

TOP = 1.7e36  # 32 * 6 * TOP = 3.26e38, below 2^128


def _scales(L, g, up, down):
    """Scale bytes of gate, up and down, in every record."""
    n = L.d * L.f
    at = 3 * n // 2
    for i, s in enumerate((g, up, down)):
        L.recs[:, at + i * n // 32:at + (i + 1) * n // 32] = s
    L.drecs = L.recs.cuda()


# rows' form, matrix form
@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (40, 4, 2)])
def test_largest_x(T, E, k):
    torch = torch_mod()
    _say("moe range, x", T, E, k)
    L = Layer(T, 256, 128, E, k, "mxfp4", 51)
    L.x = ((torch.rand(T, 256, generator=L.g) * 2 - 1) * TOP).to(torch.bfloat16)
    L.x[0] = TOP * (1 - 2.0 ** -8)
    L.dx.copy_(L.x)
    L.wr = (L.wr.float() * 2.0 ** -120).to(torch.bfloat16)  # logits of a few units
    L.dwr = L.wr.cuda()
    _scales(L, 127 - 124, 127 - 124, 121)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    L.check(b, "fp32")
    assert torch.isfinite(b["y"]).all() and b["y"].abs().max() > 0


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (40, 4, 2)])
def test_largest_h(T, E, k):
    """a and u of some 1e17: SiLU is a or nothing, to far less than their rounding."""
    torch = torch_mod()
    _say("moe range, h", T, E, k)
    d, f = 256, 128
    L = Layer(T, d, f, E, k, "mxfp4", 53)
    L.x = (L.x.float() * 2.0 ** 57).to(torch.bfloat16)
    L.dx.copy_(L.x)
    L.wr = (L.wr.float() * 2.0 ** -57).to(torch.bfloat16)
    L.dwr = L.wr.cuda()
    _scales(L, 122, 122, 127 - 120)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    torch.cuda.synchronize()
    assert torch.isfinite(b["y"]).all()
    idx, gates = (b[n].cpu() for n in ("idx", "gates"))
    want = torch.zeros(T, d, dtype=torch.float64)
    err, top, h_top = torch.zeros_like(want), torch.zeros_like(want), 0.0
    for e in idx.unique().tolist():
        ts, js = (idx == e).nonzero(as_tuple=True)
        w = [R.exactly(m) for m in M.split(L.recs[e], d, f, "mxfp4")]
        xp = R.exactly(L.x[ts])
        a, u = R.mm(xp, R.t_(w[0])), R.mm(xp, R.t_(w[1]))
        s = a[0].clamp(min=0.0), 1.2 * a[1] + 20 * R.F32 * a[0].abs() + 0.3  # |silu(a) - max(a, 0)| < 0.28
        h = R.mul(s, u)
        h_top = max(h_top, h[0].abs().max().item())
        v, c = R.mm(h, R.t_(w[2]))
        g = gates[ts, js].double()[:, None]
        want[ts] += g * v
        err[ts] += g * c
        top[ts] += g * (v.abs() + c)
    assert 1e35 < h_top < TOP
    R.check(b["y"], (want, err + (k + 1) * R.F32 * top), "y")
