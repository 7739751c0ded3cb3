"""Refusals and sizes of the routed layer for a few tokens (no GPU: every check comes before a launch)."""
import pytest

from moe_expert_offload_amd import ft

A = 1 << 20  # an aligned address; nothing below reaches a launch
BIG = 1 << 40


def _shape(E=8, d=256, f=128, k=2, fmt=ft.FT_W_BF16):
    return ft.make_shape(1, E, d, f, k, fmt)


ARGS = dict(shape=_shape(), x=A, T=2, w_router=A, allowed=None, records=A, n_slots=8, slot_of=None, residual=None, y=A,
            y_dtype=ft.FT_T_BF16, idx=A, gates=A, workspace=A, workspace_bytes=BIG)


def _fails(status, **bad):
    with pytest.raises(ft.FtError) as e:
        ft.ft_moe_layer(**{**ARGS, **bad}, stream=0)
    assert e.value.status == status, e.value
    assert ft.ft_last_error()


@pytest.mark.parametrize("bad", [
    dict(shape=_shape(d=250)), dict(shape=_shape(k=9, E=16)), dict(shape=_shape(k=3, E=2)), dict(shape=_shape(E=1025), n_slots=1025),
    dict(shape=_shape(d=264, fmt=ft.FT_W_I8)), dict(shape=_shape(d=128, fmt=ft.FT_W_MXFP4)), dict(shape=_shape(fmt=3)),
    dict(shape=_shape(d=16392)), dict(shape=_shape(d=16384, f=32768)), dict(T=-1), dict(T=65), dict(y_dtype=ft.FT_T_FP16),
    dict(n_slots=7), dict(n_slots=-1, slot_of=A), dict(x=None), dict(x=A + 8), dict(w_router=None), dict(w_router=A + 8),
    dict(records=None), dict(records=A + 8), dict(y=None), dict(y=A + 1), dict(y=A + 2, y_dtype=ft.FT_T_FP32), dict(residual=A + 1),
    dict(idx=None), dict(idx=A + 2), dict(gates=None), dict(gates=A + 2), dict(slot_of=A + 2), dict(workspace=None),
    dict(workspace=A + 16),
])
def test_refuses(bad):
    _fails(ft.FT_EINVAL, **bad)


@pytest.mark.parametrize("fmt", [ft.FT_W_BF16, ft.FT_W_MXFP4, ft.FT_W_I8])
def test_sizes(fmt):
    s = _shape(fmt=fmt)
    sizes = [ft.ft_moe_layer_workspace_bytes(s, T) for T in range(65)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert sizes[5] >= 5 * 8 * 4 + 5 * 2 * 128 * (3 if fmt == ft.FT_W_I8 else 4)
    assert ft.ft_moe_layer_workspace_bytes(s, 65) == 0 and ft.ft_moe_layer_workspace_bytes(s, -1) == 0
    _fails(ft.FT_ENOMEM, shape=s, workspace_bytes=sizes[2] - 257)
    # no tokens: nothing to do
    ft.ft_moe_layer(**{**ARGS, "shape": s, "T": 0, "x": None, "y": None, "workspace": None, "workspace_bytes": 0}, stream=0)


def test_records_of_8_bits():
    assert ft.ft_record_bytes(_shape(d=48, f=32, fmt=ft.FT_W_I8)) == 3 * 48 * 32 + 4 * (2 * 32 + 48)
    assert ft.ft_record_bytes(_shape(d=40, f=32, fmt=ft.FT_W_I8)) == 0
    assert ft.ft_record_bytes(_shape(d=48, f=24, fmt=ft.FT_W_I8)) == 0
    # a context does not take them
    s = _shape(fmt=ft.FT_W_I8)
    assert ft.ft_workspace_bytes(s, 4) == 0
    with pytest.raises(ft.FtError) as e:
        ft.ft_create(s, ft.make_config(T_max=4), n_slots=16)
    assert e.value.status == ft.FT_EUNSUPPORTED
