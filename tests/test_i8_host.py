"""Refusals and sizes of the products in 8-bit integers (no GPU: every check comes before a launch),
and pins of the plain forms their GPU tests compare against."""
import pytest
import torch

from moe_expert_offload_amd import ft
from tests import i8_ref as I8

A = 1 << 20  # an aligned address; nothing below reaches a launch
BIG = 1 << 40


def _fails(status, fn, *a, **k):
    with pytest.raises(ft.FtError) as e:
        fn(*a, **k, stream=0)
    assert e.value.status == status, e.value
    assert ft.ft_last_error()


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=2 ** 31 - 511), dict(n=0), dict(n=24), dict(n=65552), dict(dtype=ft.FT_T_FP32), dict(ld=56),
    dict(ld=68), dict(ld=1 << 22), dict(src=None), dict(src=A + 8), dict(codes=None), dict(codes=A + 8), dict(scales=None),
    dict(scales=A + 2),
])
def test_quant_refuses(bad):
    a = dict(src=A, ld=64, rows=2, n=64, dtype=ft.FT_T_BF16, codes=A, scales=A)
    _fails(ft.FT_EINVAL, ft.ft_i8_quant, **{**a, **bad})


def _m(N=24, K=64, codes=A, scales=A):
    return ft.make_i8_matrix(codes, scales, N, K)


@pytest.mark.parametrize("w", [dict(N=0), dict(N=2 ** 26 - 255), dict(K=0), dict(K=72), dict(K=65552), dict(codes=None),
                               dict(scales=None), dict(codes=A + 8), dict(scales=A + 2)])
def test_matrices_refused(w):
    _fails(ft.FT_EINVAL, ft.ft_i8_gemm, A, 64, None, 1, ft.FT_T_BF16, _m(**w), None, 24, A, 24, ft.FT_T_BF16, A, BIG)


GEMM = dict(x=A, ldx=64, x_scales=None, T=2, dtype=ft.FT_T_BF16, w=_m(), residual=None, ldr=24, y=A, ldy=24,
            y_dtype=ft.FT_T_BF16, workspace=A, workspace_bytes=BIG)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=2 ** 31 - 511), dict(T=2 ** 30, w=_m(N=128), ldy=128), dict(dtype=ft.FT_T_FP32), dict(x=None), dict(x=A + 8), dict(ldx=56), dict(ldx=70),
    dict(x_scales=A, ldx=72), dict(x_scales=A + 2), dict(y=None), dict(y=A + 1), dict(ldy=23), dict(y_dtype=ft.FT_T_FP16),
    dict(residual=A + 1), dict(residual=A + 64, ldr=8), dict(residual=A, ldr=25), dict(workspace=None),
    dict(workspace=A + 16), dict(y_dtype=ft.FT_T_FP32, y=A + 2),
])
def test_gemm_refuses(bad):
    _fails(ft.FT_EINVAL, ft.ft_i8_gemm, **{**GEMM, **bad})


def test_gemm_sizes():
    assert ft.ft_i8_gemm_workspace_bytes(-1, 8, 64, 0) == 0 and ft.ft_i8_gemm_workspace_bytes(4, 8, 60, 0) == 0
    assert ft.ft_i8_gemm_workspace_bytes(4, 0, 64, 0) == 0
    need = ft.ft_i8_gemm_workspace_bytes(2, 24, 64, 0)
    assert need >= 2 * 64 + 8 and ft.ft_i8_gemm_workspace_bytes(2, 24, 64, 1) < need
    _fails(ft.FT_ENOMEM, ft.ft_i8_gemm, **{**GEMM, "workspace_bytes": 2 * 64})
    ft.ft_i8_gemm(**{**GEMM, "T": 0, "x": None, "y": None, "workspace": None, "workspace_bytes": 0}, stream=0)
    # a workspace for the largest batch serves every smaller one
    for N, K in ((4096, 2048), (1000, 64), (65, 11008)):
        sizes = [ft.ft_i8_gemm_workspace_bytes(T, N, K, 0) for T in (0, 1, 16, 64, 65, 300, 512, 700, 2048, 8192, 16385, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_gated_ffn_refuses():
    up, down = _m(N=96, K=64), _m(N=64, K=96)
    a = dict(x=A, ldx=64, T=1, dtype=ft.FT_T_BF16, act=ft.FT_ACT_SILU, gate=up, up=up, down=down, residual=None, ldr=64,
             y=A, ldy=64, y_dtype=ft.FT_T_BF16, workspace=A, workspace_bytes=BIG)
    for bad in (dict(up=_m(N=64, K=64)), dict(down=_m(N=64, K=64)), dict(down=_m(N=96, K=96)), dict(act=5),
                dict(gate=_m(N=24, K=64), up=_m(N=24, K=64), down=_m(N=64, K=24)), dict(workspace=None),
                dict(workspace=A + 16), dict(T=-2), dict(T=2 ** 31 - 1), dict(x=None), dict(ldx=56), dict(ldy=60),
                dict(residual=A + 2, y_dtype=ft.FT_T_FP32), dict(dtype=3)):
        _fails(ft.FT_EINVAL, ft.ft_i8_gated_ffn, **{**a, **bad})
    need = ft.ft_i8_gated_ffn_workspace_bytes(1, 64, 96)
    assert need >= 96 * 3 + 4 and ft.ft_i8_gated_ffn_workspace_bytes(1, 64, 90) == 0
    _fails(ft.FT_ENOMEM, ft.ft_i8_gated_ffn, **{**a, "workspace_bytes": 128})
    ft.ft_i8_gated_ffn(**{**a, "T": 0, "x": None, "y": None, "workspace": None, "workspace_bytes": 0}, stream=0)


def test_plain_quant_on_borders():
    """127 puts the scale at 1: halves are ties, to even."""
    x = torch.tensor([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5, 0.25, 126.5, -126.5, 0, -127, 1, 2, 3]], dtype=torch.bfloat16)
    q, s = I8.quant(x)
    assert s.item() == 1.0
    assert q.tolist() == [[127, 0, 2, 2, 0, -2, -2, 64, 0, 126, -126, 0, -127, 1, 2, 3]]
    q, s = I8.quant(torch.tensor([[0.0] * 16, [float("inf")] + [1.0] * 15, [float("nan")] * 16]))
    assert q.abs().sum() == 0 and s[0] == 0 and torch.isnan(s[1:]).all()


def test_plain_quant_near_borders():
    """Codes are nearest by whole-number arithmetic: x, s as multiples of a power of two."""
    from fractions import Fraction
    g = torch.Generator().manual_seed(5)
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn(40, 64, generator=g).to(dt)
        q, s = I8.quant(x)
        for r in range(40):
            f = Fraction(s[r].item())
            for c in range(64):
                want = round(Fraction(x[r, c].item()) / f)  # ties to even
                assert want == q[r, c].item()


def test_plain_block_bound_is_tight_without_flips():
    """Whole-number rows leave one value for each element of h."""
    _, _, val, lo, hi = I8.h_values((torch.tensor([[127.0, 3.0, -5.0, 0.0]], dtype=torch.float64),
                                     torch.full((1, 4), 1e-9, dtype=torch.float64)), torch.bfloat16)
    assert torch.equal(val, lo) and torch.equal(val, hi)
