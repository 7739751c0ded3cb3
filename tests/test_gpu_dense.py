"""GPU tests of the dense operators against plain forms in 64 bits, through the C ABI.

Tolerances are the elementwise bounds of tests/dense_ref.py, derived from the number of terms,
their magnitudes and the documented roundings.
"""
import math

import pytest

from moe_expert_offload_amd import ft
from tests import dense_ref as R
from tests.gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, flush=True)


def _dt(t):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[t]


FT = {"bf16": ft.FT_T_BF16, "fp16": ft.FT_T_FP16, "fp32": ft.FT_T_FP32}
ACT = {"silu": ft.FT_ACT_SILU, "gelu": ft.FT_ACT_GELU_TANH}
SAVE = {"none": ft.FT_SAVE_NONE, "16": ft.FT_SAVE_16, "mx8": ft.FT_SAVE_MX8}


class Block:
    """A gated block's weights and calls on the GPU."""

    def __init__(self, T, d, f, t, kind, seed=0):
        torch = torch_mod()
        self.T, self.d, self.f, self.t, self.kind, self.dt = T, d, f, t, kind, _dt(t)
        self.g = torch.Generator().manual_seed(1000003 * seed + T * 7919 + d * 31 + f)
        self.wg, self.wu = self.rnd(f, d, std=d ** -0.5), self.rnd(f, d, std=d ** -0.5)
        self.wd = self.rnd(d, f, std=f ** -0.5)
        self.x, self.dy = self.rnd(T, d), self.rnd(T, d, std=0.3)

    def rnd(self, *shape, std=1.0):
        torch = torch_mod()
        return (torch.randn(*shape, generator=self.g) * std).to(self.dt).cuda()

    def forward(self, save="none", res=None, y_t=None, x=None, ldx=None, y=None, ldy=None, ldr=None, stream=None):
        torch = torch_mod()
        y_t = y_t or self.t
        if y is None:
            y = torch.full((self.T, self.d), 7.0, dtype=_dt(y_t), device="cuda")
        n = ft.ft_gated_ffn_saved_bytes(self.T, self.f, SAVE[save])
        saved = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") if save != "none" else None
        wsb = ft.ft_gated_ffn_workspace_bytes(self.T, self.d, self.f)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        self.ws = ws
        ft.ft_gated_ffn(self.x if x is None else x, ldx or self.d, self.T, self.d, self.f, FT[self.t], ACT[self.kind],
                        self.wg, self.wu, self.wd, res, ldr or self.d, y, ldy or self.d, FT[y_t], saved, SAVE[save],
                        ws, wsb, stream)
        return y, saved

    def backward(self, saved, save, x=None, x_scales=None, want_dx=True, want_dw=True, stream=None):
        torch = torch_mod()
        dx = torch.full((self.T, self.d), 7.0, dtype=self.dt, device="cuda") if want_dx else None
        dws = [torch.full_like(w, 7.0) for w in (self.wg, self.wu, self.wd)] if want_dw else [None] * 3
        wsb = ft.ft_gated_ffn_bwd_workspace_bytes(self.T, self.d, self.f, SAVE[save], x_scales is not None)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        self.ws_b = ws
        ft.ft_gated_ffn_bwd(self.x if x is None else x, self.d, x_scales, self.T, self.d, self.f, FT[self.t],
                            ACT[self.kind], self.wg, self.wu, self.wd, saved, SAVE[save], self.dy, self.d, dx, self.d,
                            *dws, ws, wsb, stream)
        return dx, *dws

    def split16(self, saved):
        n = self.T * self.f * 2
        return tuple(saved[i * n:(i + 1) * n].view(self.dt).reshape(self.T, self.f) for i in range(2))

    def split8(self, saved):
        n, m = self.T * self.f, self.T * (self.f // 32)
        c = [saved[i * n:(i + 1) * n].reshape(self.T, self.f) for i in range(2)]
        s = [saved[2 * n + i * m:2 * n + (i + 1) * m].reshape(self.T, self.f // 32) for i in range(2)]
        return c, s

    def exact(self, on="cpu"):
        return [R.exactly(v, on) for v in (self.x, self.wg, self.wu, self.wd)]


FWD = [
    # T, d, f, type, activation, save, residual, y
    (1, 8, 8, "bf16", "silu", "none", False, "bf16"),         # the smallest call
    (1, 136, 200, "fp16", "gelu", "none", True, "fp32"),
    (1, 2048, 768, "bf16", "silu", "none", False, "fp32"),    # one token at the 40-layer stack's sizes
    (13, 264, 40, "bf16", "silu", "none", True, "bf16"),
    (16, 512, 96, "fp16", "silu", "none", False, "fp16"),
    (17, 72, 104, "bf16", "gelu", "none", True, "bf16"),      # two tiles of 16 tokens
    (33, 1032, 24, "bf16", "silu", "none", False, "bf16"),    # four
    (64, 96, 520, "fp16", "silu", "none", True, "fp16"),
    (65, 96, 520, "bf16", "silu", "none", True, "fp32"),      # tiles
    (1, 64, 64, "bf16", "silu", "16", False, "bf16"),         # tiles for one token, when a and u are kept
    (3, 40, 96, "fp16", "gelu", "mx8", True, "fp16"),
    (127, 200, 136, "bf16", "gelu", "16", False, "bf16"),
    (129, 136, 160, "bf16", "silu", "mx8", True, "bf16"),
    (300, 520, 776, "fp16", "silu", "16", False, "fp16"),
    (4100, 136, 1056, "bf16", "silu", "mx8", False, "bf16"),  # large tiles, both products in turn
    (4100, 2056, 72, "fp16", "gelu", "16", True, "fp16"),
]


@pytest.mark.parametrize("T,d,f,t,kind,save,res,y_t", FWD)
def test_forward(T, d, f, t, kind, save, res, y_t):
    torch = torch_mod()
    _say("ffn", T, d, f, t, kind, save, res, y_t)
    b = Block(T, d, f, t, kind)
    r = torch.randn(T, d, generator=b.g).to(_dt(y_t)).cuda() if res else None
    y, saved = b.forward(save, r, y_t)
    torch.cuda.synchronize()
    want = R.ffn(*b.exact(), kind, b.dt, R.exactly(r) if res else None, _dt(y_t))
    R.check(y, want["y"], "y")
    if save == "16":
        for v, k in zip(b.split16(saved), "au"):
            R.check(v, R.rounded(want[k], b.dt), k)
    if save == "mx8":
        for c, s, k in zip(*b.split8(saved), "au"):
            v, e = want[k]
            step = torch.tensor([2.0 ** (i - 137) for i in range(256)], dtype=torch.float64)[s.cpu().long()]
            step = step.repeat_interleave(32, 1)  # half a step of the smallest codes
            R.check(R.mx8_values(c, s), (v, e + torch.maximum(step, 2.0 ** -4 * (v.abs() + e))), k)
            # the scale is the least that holds the block (within what the sums may be off)
            top, off = (q.reshape(T, f // 32, 32) for q in (v.abs(), e))
            got = 448 * torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64)[s.cpu().long()]
            assert ((top - off).amax(-1) <= got).all()
            assert ((top + off).amax(-1) > got / 2).all()


BWD = [
    # T, d, f, type, activation, save, x in 8 bits
    (1, 8, 8, "bf16", "silu", "16", False),
    (1, 64, 96, "fp16", "gelu", "mx8", True),
    (5, 40, 72, "bf16", "gelu", "none", False),
    (64, 96, 64, "fp16", "silu", "none", True),
    (65, 136, 200, "bf16", "silu", "16", False),        # k beyond a stage by one row
    (127, 264, 96, "bf16", "gelu", "mx8", False),
    (193, 96, 264, "fp16", "silu", "16", True),
    (300, 520, 776, "bf16", "silu", "none", False),
    (4100, 136, 2080, "bf16", "silu", "mx8", False),    # large tiles: dh
    (4100, 2080, 72, "bf16", "silu", "16", True),       # dx
    (75, 2080, 4104, "fp16", "gelu", "16", False),      # the weights' gradients
    (4100, 136, 2080, "bf16", "silu", "none", False),   # a and u again on large tiles
    (1300, 1032, 1544, "fp16", "gelu", "none", False),  # and on shared ones
]


@pytest.mark.parametrize("T,d,f,t,kind,save,x8", BWD)
def test_backward(T, d, f, t, kind, save, x8):
    torch = torch_mod()
    _say("bwd", T, d, f, t, kind, save, x8)
    b = Block(T, d, f, t, kind, seed=1)
    x, xs = b.x, None
    if x8:
        x = torch.empty((T, d), dtype=torch.uint8, device="cuda")
        xs = torch.empty((T, d // 32), dtype=torch.uint8, device="cuda")
        ft.ft_act8_pack(b.x, d, T, d, FT[t], x, xs)
    saved = None
    if save != "none":
        _, saved = b.forward(save)
    got = b.backward(saved, save, x, xs)
    torch.cuda.synchronize()
    X = (R.mx8_values(x, xs), torch.zeros(T, d, dtype=torch.float64)) if x8 else R.exactly(b.x)
    Wg, Wu, Wd = (R.exactly(w) for w in (b.wg, b.wu, b.wd))
    if save == "16":
        A, U = (R.exactly(v) for v in b.split16(saved))
    elif save == "mx8":
        A, U = ((v, torch.zeros_like(v)) for v in (R.mx8_values(c, s) for c, s in zip(*b.split8(saved))))
    else:
        A, U = (R.mm(X, R.t_(w)) for w in (Wg, Wu))
    want = R.ffn_bwd(X, Wg, Wu, Wd, A, U, R.exactly(b.dy), kind, b.dt)
    for g, k in zip(got, ("dx", "dwg", "dwu", "dwd")):
        R.check(g, want[k], k)


@pytest.mark.parametrize("T,d,f,t,res", [
    (1100, 2056, 11008, "bf16", True),   # every tile of the second product into several parts, ragged ends
    (2053, 4096, 11008, "fp16", False),  # two tiles into three parts, and an odd tile left over
    (2816, 4096, 11008, "bf16", False),  # three into four
])
def test_forward_with_shared_tiles(T, d, f, t, res):
    torch = torch_mod()
    _say("ffn shared", T, d, f, t, res)
    b = Block(T, d, f, t, "silu", seed=11)
    r = torch.randn(T, d, generator=b.g).cuda() if res else None
    y, _ = b.forward("none", r, "fp32" if res else t)
    again, _ = b.forward("none", r, "fp32" if res else t)
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    R.check(y, R.ffn(*b.exact("cuda"), "silu", b.dt, R.exactly(r, "cuda") if res else None,
                     torch.float32 if res else b.dt)["y"], "y")


@pytest.mark.parametrize("T,d,f,t", [
    (1021, 2048, 5632, "fp16"),  # dx's few tiles into four parts, across the two weights
    (8200, 2048, 4096, "bf16"),  # ragged rows' tiles into four and sixteen, behind whole ones
])
def test_backward_with_shared_tiles(T, d, f, t):
    torch = torch_mod()
    _say("bwd shared", T, d, f, t)
    b = Block(T, d, f, t, "silu", seed=12)
    _, saved = b.forward("16")
    got = b.backward(saved, "16")
    again = b.backward(saved, "16")
    torch.cuda.synchronize()
    A, U = (R.exactly(v, "cuda") for v in b.split16(saved))
    want = R.ffn_bwd(*b.exact("cuda"), A, U, R.exactly(b.dy, "cuda"), "silu", b.dt)
    for g, h, k in zip(got, again, ("dx", "dwg", "dwu", "dwd")):
        assert torch.equal(g, h)
        R.check(g, want[k], k)


def test_offsets_past_32_bits():
    """x, y, dy and dx of more than 2^31 elements: rows beyond that place, of the outputs and as the only
    ones that the weights' gradients see."""
    torch = torch_mod()
    T, d, f, n = 270000, 8192, 8, 100
    assert T * d > 2 ** 31 and (T - n) * d > 2 ** 31
    b = Block(n, d, f, "bf16", "silu", seed=13)
    x = torch.zeros((T, d), dtype=b.dt, device="cuda")
    dy = torch.zeros((T, d), dtype=b.dt, device="cuda")
    x[-n:], dy[-n:] = b.x, b.dy
    want = R.ffn(*b.exact(), "silu", b.dt)["y"]
    A, U = (R.mm(R.exactly(b.x), R.t_(R.exactly(w))) for w in (b.wg, b.wu))
    grads = R.ffn_bwd(*b.exact(), A, U, R.exactly(b.dy), "silu", b.dt)
    small = b.dy
    b.T, b.x, b.dy = T, x, dy
    y, _ = b.forward()
    torch.cuda.synchronize()
    R.check(y[-n:], want, "y")
    assert not y[:-n].any()
    del y
    got = b.backward(None, "none")
    torch.cuda.synchronize()
    R.check(got[0][-n:], grads["dx"], "dx")
    assert not got[0][:-n].any()
    for g, k in zip(got[1:], ("dwg", "dwu", "dwd")):
        R.check(g, grads[k], k)
    del small


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradients_against_differences(kind):
    """The gradients against central differences of the plain forward in 64 bits, along random
    directions; a difference of step s is off by s^2 / 6 of the third derivative (s = 1e-4: below
    1e-6 here), so what is left is the 16-bit roundings of the gradients' own bounds."""
    torch = torch_mod()
    T, d, f = 40, 64, 96
    b = Block(T, d, f, "bf16", kind, seed=2)
    got = b.backward(None, "none")
    torch.cuda.synchronize()
    X, Wg, Wu, Wd = (v[0] for v in b.exact())
    dy = b.dy.cpu().double()

    def loss(x, wg, wu, wd):
        a, u = x @ wg.t(), x @ wu.t()
        if kind == "silu":
            h = a * torch.sigmoid(a) * u
        else:
            h = torch.nn.functional.gelu(a, approximate="tanh") * u
        return ((h @ wd.t()) * dy).sum().item()

    A, U = (R.mm(R.exactly(b.x), R.t_(R.exactly(w))) for w in (b.wg, b.wu))
    bounds = R.ffn_bwd(*b.exact(), A, U, R.exactly(b.dy), kind, b.dt)
    base = [X, Wg, Wu, Wd]
    for i, k in enumerate(("dx", "dwg", "dwu", "dwd")):
        for _ in range(3):
            v = torch.randn(base[i].shape, generator=b.g).double()
            plus, minus = list(base), list(base)
            s = 1e-4
            plus[i], minus[i] = base[i] + s * v, base[i] - s * v
            diff = (loss(*plus) - loss(*minus)) / (2 * s)
            along = (got[i].cpu().double() * v).sum().item()
            room = (bounds[k][1] * v.abs()).sum().item() + 1e-6 * (bounds[k][0].abs() * v.abs()).sum().item()
            assert abs(diff - along) <= room, (k, diff, along, room)


def test_strides_and_rows_outside_stay():
    """Row strides beyond the rows, the residual in place, and what lies outside T rows and d columns untouched."""
    torch = torch_mod()
    for T, save in ((5, "none"), (100, "16"), (100, "none")):
        _say("strides", T, save)
        d, f, ldx, ldy = 72, 96, 88, 104
        b = Block(T, d, f, "bf16", "silu", seed=3)
        xw = torch.full((T + 3, ldx), float("nan"), dtype=b.dt, device="cuda")
        xw[:T, :d] = b.x
        yw = torch.randn(T + 3, ldy, generator=b.g).to(b.dt).cuda()
        before = yw.clone()
        y, saved = b.forward(save, yw, "bf16", x=xw, ldx=ldx, y=yw, ldy=ldy, ldr=ldy)
        torch.cuda.synchronize()
        want = R.ffn(*b.exact(), "silu", b.dt, R.exactly(before[:T, :d]), b.dt)
        R.check(yw[:T, :d], want["y"], "y in place")
        assert torch.equal(yw[T:], before[T:]) and torch.equal(yw[:T, d:], before[:T, d:])
    # backward
    T, d, f, ld = 70, 72, 96, 80
    b = Block(T, d, f, "fp16", "silu", seed=4)
    plain = b.backward(None, "none")
    xw, dyw = (torch.full((T + 2, ld), float("nan"), dtype=b.dt, device="cuda") for _ in range(2))
    xw[:T, :d], dyw[:T, :d] = b.x, b.dy
    dxw = torch.full((T + 2, ld), 3.0, dtype=b.dt, device="cuda")
    dws = [torch.empty_like(w) for w in (b.wg, b.wu, b.wd)]
    wsb = ft.ft_gated_ffn_bwd_workspace_bytes(T, d, f, ft.FT_SAVE_NONE, False)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ft.ft_gated_ffn_bwd(xw, ld, None, T, d, f, FT["fp16"], ACT["silu"], b.wg, b.wu, b.wd, None, ft.FT_SAVE_NONE, dyw, ld,
                        dxw, ld, *dws, ws, wsb)
    torch.cuda.synchronize()
    assert torch.equal(dxw[:T, :d], plain[0])
    assert (dxw[T:] == 3).all() and (dxw[:, d:] == 3).all()
    assert all(torch.equal(p, q) for p, q in zip(plain[1:], dws))


def test_no_rows_and_parts_not_wanted():
    torch = torch_mod()
    b = Block(0, 64, 96, "bf16", "silu")
    b.forward()
    got = b.backward(None, "none")
    torch.cuda.synchronize()
    assert all((g == 0).all() for g in got[1:])  # sums over no rows
    b = Block(50, 64, 96, "bf16", "silu", seed=5)
    full = b.backward(None, "none")
    dx = b.backward(None, "none", want_dw=False)
    dw = b.backward(None, "none", want_dx=False)
    torch.cuda.synchronize()
    assert torch.equal(dx[0], full[0]) and all(torch.equal(p, q) for p, q in zip(dw[1:], full[1:]))


def test_not_finite_rows_stay_apart():
    """A NaN or an infinity in one row reaches that row of y and dx alone."""
    torch = torch_mod()
    for T in (9, 130):
        b = Block(T, 64, 96, "bf16", "silu", seed=6)
        clean = b.forward("none")[0].clone()
        cdx = b.backward(None, "none", want_dw=False)[0].clone()
        b.x[3, 5], b.x[4, 63] = float("nan"), float("inf")
        y = b.forward("none")[0]
        dx = b.backward(None, "none", want_dw=False)[0]
        torch.cuda.synchronize()
        rest = [i for i in range(T) if i not in (3, 4)]
        assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], cdx[rest])
        assert torch.isnan(y[3]).all() and torch.isnan(dx[3]).all()
        assert not torch.isfinite(y[4]).any()


def test_extreme_gates():
    """Gates far outside exp's range: silu and its slope go to 0 and z without NaN."""
    torch = torch_mod()
    d = f = 32
    for kind in ("silu", "gelu"):
        b = Block(64, d, f, "bf16", kind, seed=7)
        b.wg.copy_(torch.eye(f, d) * 1.0)
        b.x.copy_(torch.randn(64, d, generator=b.g) * 300)
        y, saved = b.forward("16")
        got = b.backward(saved, "16")
        torch.cuda.synchronize()
        R.check(y, R.ffn(*b.exact(), kind, b.dt)["y"], "y")
        A, U = (R.exactly(v) for v in b.split16(saved))
        want = R.ffn_bwd(*b.exact(), A, U, R.exactly(b.dy), kind, b.dt)
        for g, k in zip(got, ("dx", "dwg", "dwu", "dwd")):
            R.check(g, want[k], k)


def test_largest_gates():
    """Gates up to the type's end, whose squares and cubes pass fp32: the activation is z or 0 and its
    slope 1 or 0 there, the same for both kinds, kept or computed again."""
    torch = torch_mod()
    T, d, f = 70, 32, 96
    out = {}
    for kind in ("silu", "gelu"):
        b = Block(T, d, f, "bf16", kind, seed=8)
        b.wg.copy_(torch.eye(d).repeat(f // d, 1))
        b.wu.copy_(b.wu * 2.0 ** -60)
        top = torch.exp2(torch.randint(8, 128, (T, d), generator=b.g).float())
        b.x.copy_(torch.where(torch.rand(T, d, generator=b.g) < 0.5, top, -top))
        A, u = b.x.repeat(1, f // d), b.rnd(T, f, std=2.0 ** -60)
        saved = torch.cat([v.contiguous().view(torch.uint8).flatten() for v in (A, u)])
        got = b.backward(saved, "16"), b.backward(None, "none", want_dw=False)
        torch.cuda.synchronize()
        on = R.exactly((A > 0).to(b.dt))
        x, wg, wu, wd = b.exact()
        dh = R.mm(R.exactly(b.dy), wd)
        for g, U in zip(got, (R.exactly(u), R.mm(x, R.t_(wu)))):
            da = R.rounded(R.mul(R.mul(dh, U), on), b.dt)
            du = R.rounded(R.mul(R.mul(dh, R.exactly(A)), on), b.dt)
            v, e = R.add(R.mm(da, wg), R.mm(du, wu))
            e = e + (f + 1) * R.F32 * (da[0].abs() @ wg[0].abs() + du[0].abs() @ wu[0].abs())
            R.check(g[0], R.rounded((v, e), b.dt), f"dx {kind}")
        # not dw_up = du^T x: du reaches 2^126 and x 2^127, so that its sums pass fp32 and are NaN by rights
        out[kind] = [got[0][0], got[0][1], got[0][3], got[1][0]]
    for p, q in zip(out["silu"], out["gelu"]):
        assert torch.isfinite(p).all() and torch.equal(p, q)


# ---- 8-bit activations --------------------------------------------------------------

@pytest.mark.parametrize("rows,n,t", [(1, 32, "bf16"), (3, 32, "fp16"), (257, 96, "bf16"), (5, 4096, "fp16"),
                                      (64, 2080, "bf16"), (1, 16416, "bf16")])
def test_act8_bit_exact(rows, n, t):
    torch = torch_mod()
    _say("act8", rows, n, t)
    g = torch.Generator().manual_seed(rows * 10007 + n)
    ld = n + 16
    v = torch.randn(rows, ld, generator=g) * torch.exp2(torch.randint(-14, 10, (rows, ld), generator=g).float())
    # magnitudes on the borders between codes and at the scale rule's edge
    v[:, 0:8] = torch.tensor([1.75, -1.75, 1.0625, 1.1875, 2.0 ** -9, -(2.0 ** -10), 0.0, -0.0])
    if n >= 64:
        v[:, 32:64] = 0
    v = v.to(_dt(t)).cuda()
    codes = torch.full((rows, n), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, n // 32), 255, dtype=torch.uint8, device="cuda")
    ft.ft_act8_pack(v, ld, rows, n, FT[t], codes, scales)
    out = torch.full((rows, ld), 5.0, dtype=_dt(t), device="cuda")
    ft.ft_act8_unpack(codes, scales, rows, n, FT[t], out, ld)
    torch.cuda.synchronize()
    wc, wsc = R.mx8_pack(v[:, :n].cpu().double())
    assert torch.equal(scales.cpu(), wsc)
    assert torch.equal(codes.cpu(), wc)
    assert torch.equal(out[:, :n].cpu(), R.mx8_values(wc, wsc).to(_dt(t)))
    assert (out[:, n:] == 5).all()


def test_act8_ends_of_the_range():
    """Subnormal and largest inputs, infinities and NaN."""
    torch = torch_mod()
    for t in ("bf16", "fp16"):
        dt = _dt(t)
        top = torch.finfo(dt).max
        v = torch.zeros(5, 64)
        v[0] = torch.linspace(-top, top, 64)
        v[1] = torch.finfo(dt).tiny * torch.linspace(0, 1, 64)
        v[2] = 1.5
        v[2, 3], v[2, 40] = math.inf, math.nan
        v[3] = math.inf
        v[4, 5] = -top
        v = v.to(dt).cuda()
        codes = torch.empty((5, 64), dtype=torch.uint8, device="cuda")
        scales = torch.empty((5, 2), dtype=torch.uint8, device="cuda")
        ft.ft_act8_pack(v, 64, 5, 64, FT[t], codes, scales)
        out = torch.empty((5, 64), dtype=dt, device="cuda")
        ft.ft_act8_unpack(codes, scales, 5, 64, FT[t], out, 64)
        torch.cuda.synchronize()
        wc, wsc = R.mx8_pack(v.cpu().double())
        assert torch.equal(scales.cpu(), wsc)
        nan = (wc & 127) == 127
        assert torch.equal((codes.cpu() & 127) == 127, nan)
        assert torch.equal(codes.cpu()[~nan], wc[~nan])
        want = R.mx8_values(wc, wsc).clamp(-top, top) if t == "fp16" else R.mx8_values(wc, wsc)
        assert torch.equal(torch.isnan(out.cpu()), nan)
        assert torch.equal(out.cpu()[~nan], want.to(dt)[~nan])


# ---- 4-bit weights -------------------------------------------------------------------

def _w4(g, N, K, group, zero, t):
    torch = torch_mod()
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = ((torch.rand(N, K // group, generator=g) - 0.3) * 0.02).to(_dt(t)).cuda()
    zeros = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8).cuda() if zero else None
    return codes, scales, zeros, ft.make_w4_matrix(codes, scales, zeros, N, K, group)


W4 = [
    # T, K, N, group, zeros, type, y, residual
    (1, 32, 1, 32, False, "bf16", "fp32", False),
    (1, 4096, 100, 128, False, "bf16", "fp32", False),
    (1, 160, 33, 32, True, "fp16", "fp16", True),       # a last chunk of one group
    (1, 1088, 17, 64, True, "bf16", "bf16", True),
    (4, 192, 50, 64, False, "fp16", "fp32", True),
    (15, 384, 31, 128, True, "bf16", "fp32", False),
    (17, 2048, 40, 32, True, "bf16", "fp32", True),
    (33, 640, 19, 128, False, "fp16", "fp32", False),
    (64, 224, 48, 32, True, "fp16", "fp16", False),
    (131, 256, 35, 64, True, "bf16", "fp32", True),     # three passes over the tokens
    (2, 96, 16500, 32, True, "bf16", "fp32", False),    # a block walks over several tiles of rows
    (1, 1152, 20011, 128, False, "fp16", "fp32", True),
    (40, 160, 9000, 32, True, "bf16", "fp32", False),
    (16, 4096, 64, 32, True, "bf16", "fp32", False),    # the most of x that LDS holds
    (11, 8224, 24, 32, False, "fp16", "fp32", False),   # more than that
    (16, 40960, 20, 32, True, "bf16", "fp32", False),   # the most of scales that LDS holds
    (64, 40960, 18, 32, True, "fp16", "fp32", False),
    (3, 65536, 20, 32, True, "bf16", "fp32", False),    # more than that
    (5, 64, 40, 64, True, "bf16", "fp32", False),       # one group a row
]


@pytest.mark.parametrize("T,K,N,group,zero,t,y_t,res", W4)
def test_w4_gemv(T, K, N, group, zero, t, y_t, res):
    torch = torch_mod()
    _say("w4", T, K, N, group, zero, t, y_t, res)
    g = torch.Generator().manual_seed(T * 104729 + K * 31 + N)
    codes, scales, zeros, w = _w4(g, N, K, group, zero, t)
    ldx, ldy = K + 24, N + 3
    x = torch.full((T, ldx), float("nan")).to(_dt(t))
    x[:, :K] = torch.randn(T, K, generator=g).to(_dt(t))
    x = x.cuda()
    y = torch.randn(T + 1, ldy, generator=g).to(_dt(y_t)).cuda()
    before = y.clone()
    ft.ft_w4_gemv(x, ldx, T, FT[t], w, y if res else None, ldy, y, ldy, FT[y_t])
    torch.cuda.synchronize()
    want = R.w4_mm(R.exactly(x[:, :K]), R.w4_values(codes, scales, zeros, group), codes, scales, zeros, group)
    if res:
        want = R.add(want, R.exactly(before[:T, :N]))
    R.check(y[:T, :N], R.rounded(want, _dt(y_t)), "y")
    assert torch.equal(y[T:], before[T:]) and torch.equal(y[:T, N:], before[:T, N:])


def test_w4_every_code():
    """Every code against every zero point and lane place: one-hot rows of x read the weights back."""
    torch = torch_mod()
    for t, group in (("bf16", 32), ("fp16", 64), ("bf16", 128)):
        g = torch.Generator().manual_seed(group)
        N, K = 48, 256
        codes, scales, zeros, w = _w4(g, N, K, group, True, t)
        want = R.w4_values(codes, scales, zeros, group)
        x = torch.eye(K).to(_dt(t)).cuda()
        y = torch.empty((K, N), dtype=torch.float32, device="cuda")
        ft.ft_w4_gemv(x, K, K, FT[t], w, None, N, y, N, FT["fp32"])
        torch.cuda.synchronize()
        # one exact integer times one scale: a single fp32 rounding
        assert ((y.cpu().double() - want.t()).abs() <= 2.0 ** -24 * want.t().abs()).all()


@pytest.mark.parametrize("T,d,f,groups,zero,t,kind,res", [
    (1, 256, 384, (128, 128), False, "bf16", "silu", False),
    (3, 96, 160, (32, 32), True, "fp16", "gelu", True),
    (16, 192, 64, (64, 32), True, "bf16", "silu", True),
    (40, 128, 320, (32, 64), False, "bf16", "silu", False),
    (70, 64, 96, (64, 32), True, "fp16", "silu", True),
    (1, 64, 8224, (32, 32), True, "bf16", "silu", False),
])
def test_w4_gated_ffn(T, d, f, groups, zero, t, kind, res):
    torch = torch_mod()
    _say("w4 ffn", T, d, f, groups, zero, t, kind, res)
    g = torch.Generator().manual_seed(T * 31 + d + f)
    mats = [_w4(g, f, d, groups[0], zero, t), _w4(g, f, d, groups[0], not zero, t), _w4(g, d, f, groups[1], zero, t)]
    x = torch.randn(T, d, generator=g).to(_dt(t)).cuda()
    y = torch.randn(T, d, generator=g).to(_dt(t)).cuda()
    before = y.clone()
    wsb = ft.ft_w4_gated_ffn_workspace_bytes(T, f)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ft.ft_w4_gated_ffn(x, d, T, FT[t], ACT[kind], mats[0][3], mats[1][3], mats[2][3], y if res else None, d, y, d, FT[t],
                       ws, wsb)
    torch.cuda.synchronize()

    def prod(v, m, group):
        return R.w4_mm(v, R.w4_values(*m[:3], group), *m[:3], group)

    X = R.exactly(x)
    h = R.rounded(R.mul(R.act(prod(X, mats[0], groups[0]), kind)[0], prod(X, mats[1], groups[0])), _dt(t))
    want = prod(h, mats[2], groups[1])
    if res:
        want = R.add(want, R.exactly(before))
    R.check(y, R.rounded(want, _dt(t)), "y")


# ---- together -------------------------------------------------------------------------

def test_training_steps_from_8_bits():
    """Two steps as they are used: forward keeping a and u in 8 bits, x packed, backward from the
    checkpoint, weights updated; each step's gradients against the plain backward of what was kept."""
    torch = torch_mod()
    T, d, f = 130, 96, 160
    b = Block(T, d, f, "bf16", "silu", seed=8)
    xc = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    xs = torch.empty((T, d // 32), dtype=torch.uint8, device="cuda")
    for step in range(2):
        y, saved = b.forward("mx8")
        ft.ft_act8_pack(b.x, d, T, d, FT["bf16"], xc, xs)
        got = b.backward(saved, "mx8", xc, xs)
        torch.cuda.synchronize()
        R.check(y, R.ffn(*b.exact(), "silu", b.dt)["y"], f"y {step}")
        zero = lambda v: (v, torch.zeros_like(v))  # noqa: E731
        A, U = (zero(R.mx8_values(c, s)) for c, s in zip(*b.split8(saved)))
        want = R.ffn_bwd(zero(R.mx8_values(xc, xs)), *b.exact()[1:], A, U, R.exactly(b.dy), "silu", b.dt)
        for g, k in zip(got, ("dx", "dwg", "dwu", "dwd")):
            R.check(g, want[k], f"{k} {step}")
        for w, g in zip((b.wg, b.wu, b.wd), got[1:]):
            w -= 0.05 * g


def test_shared_expert_beside_the_routed_ones():
    """The block as a layer's shared expert: grouped FFN of the routed experts, their combine, and
    the dense block added to the combined rows in place; the same expert through both gives the same."""
    torch = torch_mod()
    from tests.gpu_helpers import dev
    import numpy as np
    T, d, f = 4, 256, 128
    b = Block(T, d, f, "bf16", "silu", seed=9)
    rec = torch.cat([b.wg.flatten(), b.wu.flatten(), b.wd.flatten()])
    offsets, perm = dev(np.array([0, T], np.int32)), dev(np.arange(T, dtype=np.int32))
    slot = dev(np.zeros(1, np.int32))
    h = torch.empty(T * f * 4, dtype=torch.uint8, device="cuda")
    out = torch.empty((T, d), dtype=torch.float32, device="cuda")
    ft.ft_grouped_ffn(b.x, T, d, f, 1, rec, slot, offsets, perm, 1, 0, 1, T, h, out, 1)
    y = torch.empty((T, d), dtype=torch.float32, device="cuda")
    gates = torch.full((T, 1), 0.5, dtype=torch.float32, device="cuda")
    ft.ft_combine(out, perm, gates, None, T, 1, d, y)
    routed = y.clone()
    # the dense call reads its weights from the same record
    at = rec.data_ptr()
    wsb = ft.ft_gated_ffn_workspace_bytes(T, d, f)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ft.ft_gated_ffn(b.x, d, T, d, f, FT["bf16"], ACT["silu"], at, at + 2 * f * d, at + 4 * f * d, y, d, y, d, FT["fp32"],
                    None, ft.FT_SAVE_NONE, ws, wsb)
    torch.cuda.synchronize()
    want = R.ffn(*b.exact(), "silu", b.dt, R.exactly(routed), torch.float32)
    R.check(y, want["y"], "y")


def test_streams_graphs_and_equal_bits():
    """On a side stream behind queued work; captured and replayed with other inputs between eager
    calls; equal calls give equal bits."""
    torch = torch_mod()
    b = Block(100, 136, 264, "bf16", "silu", seed=10)
    y0, saved0 = b.forward("16")
    y0, saved0 = y0.clone(), saved0.clone()
    g0 = [g.clone() for g in b.backward(saved0, "16")]
    keep = b.x.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(2048, 2048, device="cuda")
    b.x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-3
        b.x.copy_(keep)
        y, saved = b.forward("16", stream=side)
        got = b.backward(saved, "16", stream=side)
    side.synchronize()
    assert torch.equal(y, y0) and torch.equal(saved, saved0)
    assert all(torch.equal(p, q) for p, q in zip(got, g0))
    # capture the forward, the backward and the 4-bit product of one input buffer
    gen = torch.Generator().manual_seed(5)
    codes, scales, zeros, w = _w4(gen, 64, 136 // 32 * 32, 32, True, "bf16")
    y4 = torch.empty((100, 64), dtype=torch.float32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gsaved = b.forward("16")
        ggot = b.backward(gsaved, "16")
        ws_keep = (b.ws, b.ws_b)
        ft.ft_w4_gemv(b.x, 136, 100, FT["bf16"], w, None, 64, y4, 64, FT["fp32"])
    for i in range(4):
        b.x.copy_(torch.randn(100, 136, generator=gen).to(b.dt))
        ey, es = b.forward("16")
        eg = b.backward(es, "16")
        e4 = torch.empty_like(y4)
        ft.ft_w4_gemv(b.x, 136, 100, FT["bf16"], w, None, 64, e4, 64, FT["fp32"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, ey) and torch.equal(gsaved, es) and torch.equal(y4, e4)
        assert all(torch.equal(p, q) for p, q in zip(ggot, eg))
    del ws_keep
