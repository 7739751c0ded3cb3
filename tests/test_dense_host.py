"""Refusals of the dense operators (no GPU: every check comes before a launch), and pins of the
plain forms their GPU tests compare against."""
import math
import os
import re
import subprocess

import pytest
import torch

from moe_expert_offload_amd import build, ft
from tests import dense_ref as R

A = 1 << 20  # an aligned address; nothing below reaches a launch
BIG = 1 << 40


def _fails(status, fn, *a, **k):
    with pytest.raises(ft.FtError) as e:
        fn(*a, **k, stream=0)
    assert e.value.status == status, e.value
    assert ft.ft_last_error()


def _ffn(**k):
    a = dict(x=A, ldx=64, T=4, d=64, d_ff=96, dtype=ft.FT_T_BF16, act=ft.FT_ACT_SILU, w_gate=A, w_up=A, w_down=A,
             residual=None, ldr=64, y=A, ldy=64, y_dtype=ft.FT_T_BF16, saved=None, save_fmt=ft.FT_SAVE_NONE,
             workspace=A, workspace_bytes=BIG)
    a.update(k)
    return a


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=60), dict(d_ff=100), dict(d=1 << 21), dict(dtype=ft.FT_T_FP32), dict(dtype=7),
    dict(act=2), dict(w_gate=None), dict(w_up=A + 8), dict(w_down=A + 2), dict(x=None), dict(x=A + 8), dict(ldx=56),
    dict(ldx=68), dict(ldx=1 << 22), dict(y=None), dict(y=A + 4), dict(ldy=60), dict(y_dtype=ft.FT_T_FP16),
    dict(residual=A + 64, ldr=32), dict(residual=A + 4), dict(residual=A, ldr=72), dict(save_fmt=3),
    dict(save_fmt=ft.FT_SAVE_16), dict(save_fmt=ft.FT_SAVE_16, saved=A + 8),
    dict(save_fmt=ft.FT_SAVE_MX8, saved=A, d_ff=104), dict(workspace=None), dict(workspace=A + 16),
])
def test_gated_ffn_refuses(bad):
    _fails(ft.FT_EINVAL, ft.ft_gated_ffn, **_ffn(**bad))


def test_gated_ffn_sizes():
    need = ft.ft_gated_ffn_workspace_bytes(4, 64, 96)
    assert need >= 4 * 96 * 2
    _fails(ft.FT_ENOMEM, ft.ft_gated_ffn, **_ffn(workspace_bytes=need - 1))
    assert ft.ft_gated_ffn_workspace_bytes(-1, 64, 96) == 0 and ft.ft_gated_ffn_workspace_bytes(4, 60, 96) == 0
    assert ft.ft_gated_ffn_saved_bytes(5, 96, ft.FT_SAVE_NONE) == 0
    assert ft.ft_gated_ffn_saved_bytes(5, 96, ft.FT_SAVE_16) == 5 * 96 * 4
    assert ft.ft_gated_ffn_saved_bytes(5, 96, ft.FT_SAVE_MX8) == 2 * 5 * (96 + 3)
    assert ft.ft_gated_ffn_saved_bytes(5, 104, ft.FT_SAVE_MX8) == 0
    # no rows: nothing to do, null tensors or not
    ft.ft_gated_ffn(**_ffn(T=0, x=None, y=None, workspace=None, workspace_bytes=0), stream=0)


def _bwd(**k):
    a = dict(x=A, ldx=64, x_scales=None, T=4, d=64, d_ff=96, dtype=ft.FT_T_BF16, act=ft.FT_ACT_SILU, w_gate=A, w_up=A,
             w_down=A, saved=A, save_fmt=ft.FT_SAVE_16, dy=A, lddy=64, dx=A, lddx=64, dw_gate=A, dw_up=A, dw_down=A,
             workspace=A, workspace_bytes=BIG)
    a.update(k)
    return a


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=4), dict(d_ff=0), dict(dtype=ft.FT_T_FP32), dict(act=-1), dict(w_down=None), dict(saved=None),
    dict(saved=A + 8), dict(save_fmt=-1), dict(save_fmt=ft.FT_SAVE_MX8, d_ff=104), dict(dy=None), dict(dy=A + 8),
    dict(lddy=56), dict(lddx=60), dict(dx=A + 8), dict(dw_gate=None), dict(dw_up=None, dw_gate=None), dict(dw_down=A + 4),
    dict(x=None), dict(ldx=72, x_scales=A), dict(d=72, ldx=72, lddy=72, lddx=72, x_scales=A), dict(workspace=A + 128),
])
def test_gated_ffn_bwd_refuses(bad):
    _fails(ft.FT_EINVAL, ft.ft_gated_ffn_bwd, **_bwd(**bad))


def test_gated_ffn_bwd_sizes():
    base = ft.ft_gated_ffn_bwd_workspace_bytes(4, 64, 96, ft.FT_SAVE_16, False)
    assert base >= 4 * 96 * 6
    assert ft.ft_gated_ffn_bwd_workspace_bytes(4, 64, 96, ft.FT_SAVE_NONE, True) >= base + 4 * 96 * 4 + 4 * 64 * 2
    assert ft.ft_gated_ffn_bwd_workspace_bytes(4, 64, 96, 9, False) == 0
    _fails(ft.FT_ENOMEM, ft.ft_gated_ffn_bwd, **_bwd(workspace_bytes=base - 1))
    _fails(ft.FT_ENOMEM, ft.ft_gated_ffn_bwd, **_bwd(workspace_bytes=base, x_scales=A))
    # nothing wanted: nothing to do
    ft.ft_gated_ffn_bwd(**_bwd(dx=None, dw_gate=None, dw_up=None, dw_down=None), stream=0)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(n=16), dict(n=0), dict(dtype=ft.FT_T_FP32), dict(ld=32), dict(ld=68)])
def test_act8_refuses(bad):
    a = dict(rows=2, n=64, dtype=ft.FT_T_BF16, ld=64)
    a.update(bad)
    _fails(ft.FT_EINVAL, ft.ft_act8_pack, A, a["ld"], a["rows"], a["n"], a["dtype"], A, A)
    _fails(ft.FT_EINVAL, ft.ft_act8_unpack, A, A, a["rows"], a["n"], a["dtype"], A, a["ld"])


def test_act8_refuses_pointers():
    for i in range(3):
        for bad in (None, A + 8):
            p = [A, A, A + 1]
            p[i] = bad
            if i == 2 and bad:
                continue  # scales need no alignment
            _fails(ft.FT_EINVAL, ft.ft_act8_pack, p[0], 64, 2, 64, ft.FT_T_BF16, p[1], p[2])
            _fails(ft.FT_EINVAL, ft.ft_act8_unpack, p[1], p[2], 2, 64, ft.FT_T_BF16, p[0], 64)


def _m(N=24, K=64, group=32, codes=A, scales=A, zeros=None):
    return ft.make_w4_matrix(codes, scales, zeros, N, K, group)


@pytest.mark.parametrize("w", [
    dict(N=0), dict(K=0), dict(K=96, group=64), dict(group=16), dict(group=256, K=256), dict(codes=None),
    dict(scales=None), dict(codes=A + 8), dict(scales=A + 1),
])
def test_w4_refuses_matrices(w):
    _fails(ft.FT_EINVAL, ft.ft_w4_gemv, A, 64, 1, ft.FT_T_BF16, _m(**w), None, 24, A, 24, ft.FT_T_BF16)


@pytest.mark.parametrize("k", [
    dict(T=-1), dict(dtype=ft.FT_T_FP32), dict(x=None), dict(x=A + 2), dict(ldx=32), dict(ldx=70), dict(y=None),
    dict(y=A + 1), dict(ldy=23), dict(y_dtype=ft.FT_T_FP16), dict(residual=A + 1), dict(residual=A + 64, ldr=8),
    dict(residual=A, ldr=25),
])
def test_w4_gemv_refuses(k):
    a = dict(x=A, ldx=64, T=1, dtype=ft.FT_T_BF16, w=_m(), residual=None, ldr=24, y=A, ldy=24, y_dtype=ft.FT_T_BF16)
    a.update(k)
    _fails(ft.FT_EINVAL, ft.ft_w4_gemv, **a)


def test_w4_gated_ffn_refuses():
    up, down = _m(N=96, K=64), _m(N=64, K=96)
    a = dict(x=A, ldx=64, T=1, dtype=ft.FT_T_BF16, act=ft.FT_ACT_SILU, gate=up, up=up, down=down, residual=None, ldr=64,
             y=A, ldy=64, y_dtype=ft.FT_T_BF16, workspace=A, workspace_bytes=BIG)
    for bad in (dict(up=_m(N=64, K=64)), dict(down=_m(N=64, K=64)), dict(down=_m(N=96, K=96)), dict(up=_m(N=96, K=64, group=64)),
                dict(act=5), dict(workspace=None), dict(workspace=A + 16), dict(T=-2), dict(x=None), dict(ldx=56)):
        _fails(ft.FT_EINVAL, ft.ft_w4_gated_ffn, **{**a, **bad})
    need = ft.ft_w4_gated_ffn_workspace_bytes(1, 96)
    _fails(ft.FT_ENOMEM, ft.ft_w4_gated_ffn, **{**a, "workspace_bytes": need - 1})


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 511, 2 ** 31 - 64])
def test_rows_past_32_bits_are_refused(T):
    """Row counts whose sums with a tile's size pass 32 bits."""
    assert ft.ft_gated_ffn_workspace_bytes(T, 64, 96) == 0 and ft.ft_gated_ffn_saved_bytes(T, 96, ft.FT_SAVE_16) == 0
    assert ft.ft_gated_ffn_bwd_workspace_bytes(T, 64, 96, ft.FT_SAVE_16, False) == 0
    _fails(ft.FT_EINVAL, ft.ft_gated_ffn, **_ffn(T=T))
    _fails(ft.FT_EINVAL, ft.ft_gated_ffn_bwd, **_bwd(T=T))
    _fails(ft.FT_EINVAL, ft.ft_w4_gemv, A, 64, T, ft.FT_T_BF16, _m(), None, 24, A, 24, ft.FT_T_BF16)
    up, down = _m(N=96, K=64), _m(N=64, K=96)
    _fails(ft.FT_EINVAL, ft.ft_w4_gated_ffn, A, 64, T, ft.FT_T_BF16, ft.FT_ACT_SILU, up, up, down, None, 64, A, 64,
           ft.FT_T_BF16, A, BIG)


def test_w4_limits():
    _fails(ft.FT_EINVAL, ft.ft_w4_gemv, A, 64, 65535 * 64 + 1, ft.FT_T_BF16, _m(), None, 24, A, 24, ft.FT_T_BF16)
    n = 2 ** 27 - 15  # a grid of 2^32 threads
    _fails(ft.FT_EINVAL, ft.ft_w4_gemv, A, 64, 1, ft.FT_T_BF16, _m(N=n), None, n, A, n, ft.FT_T_BF16)


# rows at the ends of tiles, of stages and of rounds of tiles, and in between
ROWS = (1, 2, 16, 17, 63, 64, 65, 127, 128, 129, 192, 193, 256, 300, 512, 640, 700, 1000, 1021, 1024, 1300, 2048, 2053, 2816,
        4096, 4100, 4416, 4928, 5000, 7616, 8192, 8200, 11072, 16383, 16384, 16385, 20000, 65536, 270000)


@pytest.mark.parametrize("d,f", [(4096, 2048), (2048, 768), (4096, 11008), (2048, 5632), (8192, 8), (256, 512), (64, 96)])
def test_a_workspace_serves_fewer_rows(d, f):
    """No size falls as the rows grow: a buffer for the largest batch is large enough for each smaller one."""
    sizes = [lambda T: ft.ft_gated_ffn_workspace_bytes(T, d, f)]
    if f % 32 == 0:
        sizes.append(lambda T: ft.ft_w4_gated_ffn_workspace_bytes(T, f))
    sizes += [lambda T, s=s, x=x: ft.ft_gated_ffn_bwd_workspace_bytes(T, d, f, s, x)
              for s in (ft.FT_SAVE_NONE, ft.FT_SAVE_16, ft.FT_SAVE_MX8) for x in (False, True)]
    for size in sizes:
        got = [size(T) for T in ROWS]
        assert all(0 < a <= b for a, b in zip(got, got[1:])), [(T, n) for T, n in zip(ROWS, got)]


# ---- the plain forms themselves --------------------------------------------------------

def test_plain_backward_is_autograd():
    """The plain gradients equal torch's automatic ones in 64 bits."""
    g = torch.Generator().manual_seed(0)
    T, d, f = 7, 16, 24
    for kind in ("silu", "gelu"):
        x, wg, wu, wd, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in
                             ((T, d), (f, d), (f, d), (d, f), (T, d)))
        leaves = [v.clone().requires_grad_(True) for v in (x, wg, wu, wd)]
        a, u = leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t()
        fn = torch.nn.functional.silu if kind == "silu" else (lambda v: torch.nn.functional.gelu(v, approximate="tanh"))
        y = (fn(a) * u) @ leaves[3].t()
        auto = torch.autograd.grad(y, leaves, dy)
        z = lambda v: (v, torch.zeros_like(v))  # noqa: E731
        got = R.ffn_bwd(z(x), z(wg), z(wu), z(wd), z(a.detach()), z(u.detach()), z(dy), kind, torch.bfloat16)
        for k, v in zip(("dx", "dwg", "dwu", "dwd"), auto):
            assert torch.allclose(got[k][0], v, rtol=1e-12, atol=1e-12), k
        assert torch.allclose(R.ffn(z(x), z(wg), z(wu), z(wd), kind, torch.bfloat16)["y"][0], y, rtol=1e-12, atol=1e-12)


def test_bounds_hold_for_a_bf16_computation_and_catch_a_wrong_one():
    g = torch.Generator().manual_seed(1)
    T, d, f, dt = 9, 64, 48, torch.bfloat16
    x, wg, wu, wd = ((torch.randn(*s, generator=g) * k).to(dt) for s, k in (((T, d), 1), ((f, d), .1), ((f, d), .1), ((d, f), .1)))
    a, u = x.float() @ wg.float().t(), x.float() @ wu.float().t()
    h = (torch.nn.functional.silu(a) * u).to(dt)
    want = R.ffn(*(R.exactly(v) for v in (x, wg, wu, wd)), "silu", dt)["y"]
    R.check((h.float() @ wd.float().t()).to(dt), want, "y")
    wrong = (torch.nn.functional.gelu(a) * u).to(dt)
    with pytest.raises(AssertionError):
        R.check((wrong.float() @ wd.float().t()).to(dt), want, "y")


def test_mx8_rule():
    """The scale is the least power of two that holds the block, codes are the nearest points."""
    v = torch.zeros(6, 32, dtype=torch.float64)
    v[0, 0] = 448.0       # exactly the largest code at scale 1
    v[1, 0] = 448.0001    # needs scale 2
    v[2, 0], v[2, 1] = 1.0, 1.0 + 1 / 16  # a tie between 1 and 1.125 at this scale goes to the even code
    v[3, 0], v[3, 1] = 2.0 ** -130, -(2.0 ** -133)
    v[4, 0], v[4, 1] = math.inf, -3.0
    c, s = R.mx8_pack(v)
    assert s[0, 0] == 127 and c[0, 0] == 126
    assert s[1, 0] == 128 and s[2, 0] == 127 - 8
    assert R.mx8_values(c, s)[2, 1] == 1.0
    assert s[3, 0] == 0 and R.mx8_values(c, s)[3, 0] == 2.0 ** -130
    assert c[4, 0] == 127 and R.mx8_values(c, s)[4, 1] == -3.0
    assert s[5, 0] == 0 and (c[5] == 0).all()
    assert R.e4m3_points()[126] == 448 and R.e4m3_points()[8] == 2.0 ** -6
    pts = torch.arange(126, dtype=torch.uint8)
    assert torch.equal(pts.view(torch.float8_e4m3fn).double(), R.e4m3_points()[:126])


# ---- generated code --------------------------------------------------------------------

def test_hand_issued_loads_write_lds(tmp_path):
    """The tiled products load straight into LDS with inline-asm loads and count their waits by hand:
    whatever else the compiler issues only makes such a wait stricter, but an inline-asm load into a
    register could be copied before its data lands.  There is none."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path / "dense.s"
    cmd = [build.HIPCC, f"--offload-arch={build.ARCH}", "--cuda-device-only", "-S", "-O3", "-std=c++17",
           f"-I{os.path.join(build.PKG, '..', 'include')}", "-o", str(out),
           os.path.join(build.CSRC, "kernels_dense.hip")] + build.DEVICE_FLAGS
    subprocess.run(cmd, check=True, capture_output=True, timeout=600)
    src = out.read_text()
    seen = 0
    for name, body in re.findall(r"^(_Z\w*gemm(?:256)?_kernel\w*):[^\n]*\n(.*?); -- End function", src, re.S | re.M):
        blocks = re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", body, re.S)
        loads = [v.strip() for b in blocks for v in b.split("\n") if re.match(r"\s*(buffer|global|flat|scratch)_load", v)]
        assert loads and all(v.endswith(" lds") for v in loads), name
        # on entry, and in the whole and the ragged walk twice a stage (256 rows) or once (128 rows)
        if "gemm256" in name and "ELi2EE" in name:
            assert sum("s_waitcnt vmcnt(8)" in b for b in blocks) == 5, name
        elif "gemm256" in name:
            assert sum("s_waitcnt vmcnt(6)" in b for b in blocks) == 3, name
        seen += 1
    assert seen == 36  # 6 modes, 2 types, 3 tile sizes
