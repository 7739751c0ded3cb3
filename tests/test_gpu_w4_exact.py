"""GPU tests of the products with 4-bit weights on whole-number inputs whose sums are exact in fp32 (compared for
equality), at row lengths where every form loads its registers again, and of values that are not finite."""
import pytest

from moe_expert_offload_amd import ft
from tests.gpu_helpers import torch_mod
from tests.test_gpu_dense import ACT, FT, _dt, _say

pytestmark = pytest.mark.gpu


def _ints(g, lo, hi, *shape):
    torch = torch_mod()
    return torch.randint(lo, hi + 1, shape, generator=g)


def _pack(values, zeros, scales, group, t):
    """A matrix (code - zero) * scale of whole `values`, and what keeps it alive."""
    torch = torch_mod()
    N, K = values.shape
    z = torch.full((N, K // group), 8) if zeros is None else zeros
    code = values + z.repeat_interleave(group, 1)
    assert code.min() >= 0 and code.max() <= 15
    packed = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8).cuda()
    s = scales.to(_dt(t)).cuda()
    zd = None if zeros is None else zeros.to(torch.uint8).cuda()
    return (packed, s, zd), ft.make_w4_matrix(packed, s, zd, N, K, group)


GEMV = [
    # T, K, N, group, zero, type, y, residual: K past 16 (8 where few are in flight) chunks of 128 a wave
    (1, 11008, 40, 128, False, "bf16", "fp32", False),
    (2, 4256, 33, 32, True, "fp16", "fp32", True),
    (3, 4224, 50, 128, True, "bf16", "bf16", False),
    (4, 8256, 17, 64, False, "fp16", "fp32", False),
    (5, 11008, 200, 64, True, "fp16", "fp32", True),
    (8, 4256, 48, 32, False, "bf16", "fp32", False),
    (8, 4224, 31, 128, True, "bf16", "bf16", True),
    (13, 4288, 40, 64, True, "fp16", "fp32", False),
    (16, 11008, 35, 32, True, "bf16", "fp32", True),
    (17, 4224, 40, 128, False, "bf16", "fp32", False),
    (32, 6432, 50, 32, True, "fp16", "fp32", False),
    (33, 4288, 19, 64, False, "bf16", "bf16", True),
    (64, 4256, 36, 32, True, "bf16", "fp32", False),
    (70, 2304, 40, 128, True, "fp16", "fp32", True),
    (200, 1056, 24, 32, False, "bf16", "fp32", False),
    (9, 4224, 7, 128, True, "bf16", "fp32", False),      # fewer rows than a tile: scales from memory
    (6, 65536, 18, 32, True, "fp16", "fp32", False),     # more scales than LDS holds
]


@pytest.mark.parametrize("T,K,N,group,zero,t,y_t,res", GEMV)
def test_gemv_exact(T, K, N, group, zero, t, y_t, res):
    torch = torch_mod()
    _say("w4 exact", T, K, N, group, zero, t, y_t, res)
    g = torch.Generator().manual_seed(T * 7 + K + N)
    KG = K // group
    zeros = _ints(g, 0, 15, N, KG) if zero else None
    z = torch.full((N, KG), 8) if zeros is None else zeros
    values = _ints(g, 0, 15, N, K) - z.repeat_interleave(group, 1)
    scales = torch.pow(2.0, -_ints(g, 4, 6, N, KG).double())
    keep, w = _pack(values, zeros, scales, group, t)
    x = _ints(g, -3, 3, T, K).double()
    full = values.double() * scales.repeat_interleave(group, 1)
    # every partial sum is a multiple of 2^-6 below 2^18, a group's (16 + code) x below 2^24
    assert (x.abs() @ full.abs().t()).max() < 2 ** 18 and group * 31 * 3 < 2 ** 24
    r = _ints(g, -100, 100, T, N).double() if res else None
    want = x @ full.t() + (r if res else 0)
    y = (r if res else torch.full((T, N), 7.0)).to(_dt(y_t)).cuda()
    ft.ft_w4_gemv(x.to(_dt(t)).cuda(), K, T, FT[t], w, y if res else None, N, y, N, FT[y_t])
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), want.float().to(_dt(y_t)))
    del keep


@pytest.mark.parametrize("T,d,f,groups,zero,t,kind", [
    (1, 4224, 96, (128, 32), False, "bf16", "silu"),
    (3, 4256, 160, (32, 32), True, "fp16", "gelu"),
    (7, 4288, 64, (64, 64), True, "bf16", "silu"),
    (16, 4224, 128, (128, 128), False, "fp16", "silu"),
    (16, 4256, 96, (32, 32), True, "bf16", "silu"),
    (20, 4224, 96, (128, 32), True, "bf16", "gelu"),
    (40, 4256, 64, (32, 64), False, "fp16", "silu"),
    (70, 4288, 96, (64, 32), True, "bf16", "silu"),
])
def test_gated_ffn_exact(T, d, f, groups, zero, t, kind):
    """Gates of 33 and more, where both activations are the gate itself to the last bit: h is one product of whole
    numbers, rounded once.  The down matrix picks one h a row, so that y shows each of them."""
    torch = torch_mod()
    _say("w4 ffn exact", T, d, f, groups, zero, t, kind)
    g = torch.Generator().manual_seed(T + d + 3 * f)
    G = groups[0]
    mats, full = [], []
    for lo, hi in ((0, 3), (-2, 2)):
        zeros = _ints(g, 4, 11, f, d // G) if zero else None
        v = _ints(g, lo, hi, f, d)
        s = torch.pow(2.0, _ints(g, 0, 1, f, d // G).double())
        mats.append(_pack(v, zeros, s, G, t))
        full.append(v.double() * s.repeat_interleave(G, 1))
    pick = torch.arange(d) % f
    down = torch.zeros(d, f, dtype=torch.int64)
    down[torch.arange(d), pick] = 1
    zeros = _ints(g, 0, 14, d, f // groups[1]) if zero else None
    mats.append(_pack(down, zeros, torch.ones(d, f // groups[1]), groups[1], t))
    x = (torch.rand(T, d, generator=g) < 60 / d).double()
    a, u = x @ full[0].t(), x @ full[1].t()
    assert a.min() >= 33 and a.max() < 1024 and u.abs().max() < 1024
    h = (a * u).float().to(_dt(t))
    assert (31 * h.double().abs().reshape(T, -1, groups[1]).sum(-1)).max() < 2 ** 24
    y = torch.full((T, d), 7.0, dtype=_dt(t), device="cuda")
    wsb = ft.ft_w4_gated_ffn_workspace_bytes(T, f)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ft.ft_w4_gated_ffn(x.to(_dt(t)).cuda(), d, T, FT[t], ACT[kind], mats[0][1], mats[1][1], mats[2][1], None, d, y, d, FT[t],
                       ws, wsb)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), h[:, pick])


@pytest.mark.parametrize("T", [1, 3, 7, 14, 30, 50, 90])
def test_not_finite_rows_stay_apart(T):
    """An infinity or a NaN in a row of x makes that row of y NaN (the weights go through the sums in two parts) and
    leaves every other row's bits as they were; an h past fp16's end does the same to its row of the gated block."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(T)
    K, N, f, group = 1152, 40, 64, 64

    def matrix(rows, cols):
        return _pack(_ints(g, -8, 7, rows, cols), None, torch.rand(rows, cols // group, generator=g) * 0.02 + 0.01, group,
                     "fp16")

    (k0, w), (k1, up), (k2, gate), (k3, down) = matrix(N, K), matrix(f, K), matrix(f, K), matrix(K, f)
    x = torch.randn(T, K, generator=g).half()
    bad = sorted({0, T // 2, T - 1})
    y = torch.empty((2, T, N), dtype=torch.float32, device="cuda")
    z = torch.empty((2, T, K), dtype=torch.float16, device="cuda")
    wsb = ft.ft_w4_gated_ffn_workspace_bytes(T, f)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    for i in range(2):
        v = x.clone()
        if i:
            for j, r in enumerate(bad):
                v[r, 37 + 300 * j] = (float("inf"), float("nan"), -float("inf"))[j]
        ft.ft_w4_gemv(v.cuda(), K, T, FT["fp16"], w, None, N, y[i], N, FT["fp32"])
        big = x.clone()
        if i:
            big[bad] *= 4096  # a and u of thousands: h past 65504
        ft.ft_w4_gated_ffn(big.cuda(), K, T, FT["fp16"], ACT["silu"], gate, up, down, None, K, z[i], K, FT["fp16"], ws, wsb)
    torch.cuda.synchronize()
    rest = [r for r in range(T) if r not in bad]
    assert torch.isnan(y[1][bad]).all() and torch.equal(y[1][rest], y[0][rest])
    assert torch.isnan(z[1][bad]).any(1).all() and torch.equal(z[1][rest], z[0][rest])
    assert torch.isfinite(y[0]).all() and torch.isfinite(z[0]).all()
    del k0, k1, k2, k3
