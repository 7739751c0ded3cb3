"""GPU tests of the dense operators' contracts at their edges, through the C ABI."""
import pytest

from moe_expert_offload_amd import ft
from tests import dense_ref as R
from tests.gpu_helpers import torch_mod
from tests.test_gpu_dense import ACT, FT, SAVE, Block, _say

pytestmark = pytest.mark.gpu


def test_one_workspace_for_every_batch():
    """A workspace made once for the largest batch, used by falling and rising numbers of rows: nothing is
    refused, and the bits are those of a workspace of the call's own."""
    torch = torch_mod()
    d, f, t, top = 1024, 512, "bf16", 2053
    size = max(ft.ft_gated_ffn_workspace_bytes(top, d, f),
               *(ft.ft_gated_ffn_bwd_workspace_bytes(top, d, f, s, False) for s in SAVE.values()))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for T, save in ((2053, "mx8"), (512, "16"), (300, "none"), (64, "none"), (65, "16"), (1, "none"), (1, "mx8"),
                    (700, "16"), (1300, "none"), (2048, "16")):
        _say("one workspace", T, save)
        n = ft.ft_gated_ffn_workspace_bytes(top, d, f)
        nb = ft.ft_gated_ffn_bwd_workspace_bytes(top, d, f, SAVE[save], False)
        b = Block(T, d, f, t, "silu", seed=21)
        y, saved = b.forward(save)
        want = b.backward(saved, save)
        y2, saved2 = torch.empty_like(y), None if saved is None else torch.empty_like(saved)
        ft.ft_gated_ffn(b.x, d, T, d, f, FT[t], ACT["silu"], b.wg, b.wu, b.wd, None, d, y2, d, FT[t], saved2, SAVE[save],
                        ws, n)
        got = [torch.empty_like(w) for w in want]
        ft.ft_gated_ffn_bwd(b.x, d, None, T, d, f, FT[t], ACT["silu"], b.wg, b.wu, b.wd, saved2, SAVE[save], b.dy, d,
                            got[0], d, *got[1:], ws, nb)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and (saved is None or torch.equal(saved, saved2))
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_few_rows_need_no_more_than_h():
    """Up to 64 rows with nothing kept, the weights stream once and nothing is shared between blocks: h is
    all that the workspace holds, whatever the sizes."""
    torch = torch_mod()
    T, d, f, t = 3, 4096, 2048, "bf16"
    b = Block(T, d, f, t, "silu", seed=22)
    y, _ = b.forward("none")
    n = T * f * 2 + 512
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    ws[n:] = 77
    y2 = torch.empty_like(y)
    ft.ft_gated_ffn(b.x, d, T, d, f, FT[t], ACT["silu"], b.wg, b.wu, b.wd, None, d, y2, d, FT[t], None, ft.FT_SAVE_NONE, ws, n)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and (ws[n:] == 77).all()
    with pytest.raises(ft.FtError) as e:  # the same rows with a and u kept go by shared tiles
        saved = torch.empty(ft.ft_gated_ffn_saved_bytes(T, f, ft.FT_SAVE_16), dtype=torch.uint8, device="cuda")
        ft.ft_gated_ffn(b.x, d, T, d, f, FT[t], ACT["silu"], b.wg, b.wu, b.wd, None, d, y2, d, FT[t], saved, ft.FT_SAVE_16,
                        ws, n)
    assert e.value.status == ft.FT_ENOMEM


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_from_the_largest_mx8_values(kind):
    """A finite a, u or x next to the type's end is packed to 2^128, which fp32 does not hold: the backward pass takes
    the largest value there (slope 1 or 0 of both activations), not an infinity whose slope is NaN."""
    torch = torch_mod()
    T, d, f = 70, 32, 96
    b = Block(T, d, f, "bf16", kind, seed=23)
    b.dy.copy_(b.rnd(T, d, std=2.0 ** -40))
    # the whole way: the largest a's as the forward call packs them
    top = torch.finfo(torch.bfloat16).max
    x0 = torch.zeros(T, d)
    x0[:, 0] = torch.where(torch.rand(T, generator=b.g) < 0.5, top, -top)
    x0[:, 1] = 1.0
    b.x.copy_(x0)
    b.wg.zero_()
    b.wg[:, 0] = 1.0
    b.wu.zero_()
    b.wu[:, 1] = b.rnd(f, std=2.0 ** -60)
    _, saved = b.forward("mx8")
    c, s = b.split8(saved)
    torch.cuda.synchronize()
    A, U = (R.mx8_values(ci, si) for ci, si in zip(c, s))
    assert (A.abs() == 2.0 ** 128).all()
    A = A.clamp(-torch.finfo(torch.float32).max, torch.finfo(torch.float32).max)
    b.wu.copy_(b.rnd(f, d, std=d ** -0.5))
    b.x.copy_(b.rnd(T, d))
    got = b.backward(saved, "mx8")
    torch.cuda.synchronize()
    zero = lambda v: (v, torch.zeros_like(v))  # noqa: E731
    on = zero((A > 0).double())
    x, wg, wu, wd = b.exact()
    dy = R.exactly(b.dy)
    dh = R.mm(dy, wd)
    h = R.rounded(R.mul(R.mul(zero(A), on), zero(U)), b.dt)
    da = R.rounded(R.mul(R.mul(dh, zero(U)), on), b.dt)
    du = R.rounded(R.mul(R.mul(dh, zero(A)), on), b.dt)
    v, e = R.add(R.mm(da, wg), R.mm(du, wu))
    e = e + (f + 1) * R.F32 * (da[0].abs() @ wg[0].abs() + du[0].abs() @ wu[0].abs())
    R.check(got[0], R.rounded((v, e), b.dt), "dx")
    for g, w, k in zip(got[1:], (R.mm(R.t_(da), x), R.mm(R.t_(du), x), R.mm(R.t_(dy), h)), ("dwg", "dwu", "dwd")):
        R.check(g, R.rounded(w, b.dt), k)


def test_backward_from_the_largest_mx8_x():
    torch = torch_mod()
    T, d, f = 70, 64, 96
    b = Block(T, d, f, "bf16", "silu", seed=24)
    b.dy.copy_(b.rnd(T, d, std=2.0 ** -40))
    _, saved = b.forward("16")
    pick = torch.tensor([120, 248, 126, 254, 56, 3, 0], dtype=torch.uint8)  # +-256, +-448, 1, 3 * 2^-9, 0
    xc = pick[torch.randint(0, 7, (T, d), generator=b.g)].cuda()
    xs = torch.full((T, d // 32), 247, dtype=torch.uint8, device="cuda")
    got = b.backward(saved, "16", xc, xs)
    torch.cuda.synchronize()
    top = torch.finfo(torch.bfloat16).max
    X = R.mx8_values(xc, xs).clamp(-top, top)
    A, U = (R.exactly(v) for v in b.split16(saved))
    want = R.ffn_bwd((X, torch.zeros_like(X)), *b.exact()[1:], A, U, R.exactly(b.dy), "silu", b.dt)
    for g, k in zip(got, ("dx", "dwg", "dwu", "dwd")):
        R.check(g, want[k], k)


@pytest.mark.parametrize("n", [32, 96])
def test_act8_of_many_rows(n):
    """More blocks than the first dimension of a grid takes: every row is packed and unpacked once, the last ones too."""
    torch = torch_mod()
    rows = 65536 * 128 * 2 + 77
    src = torch.randint(-448, 449, (rows, n), device="cuda", dtype=torch.int16).to(torch.bfloat16)
    codes = torch.empty((rows + 1, n), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows + 1, n // 32), dtype=torch.uint8, device="cuda")
    out = torch.empty((rows + 1, n), dtype=torch.bfloat16, device="cuda")
    codes[-1], scales[-1], out[-1] = 33, 44, 55
    ft.ft_act8_pack(src, n, rows, n, FT["bf16"], codes, scales)
    ft.ft_act8_unpack(codes, scales, rows, n, FT["bf16"], out, n)
    torch.cuda.synchronize()
    assert (codes[-1] == 33).all() and (scales[-1] == 44).all() and (out[-1] == 55).all()
    for at in (0, 65536 * 128 - 1, 65536 * 128, rows - 300):
        wc, ws = R.mx8_pack(src[at:at + 300].cpu().double())
        m = wc.shape[0]
        assert torch.equal(codes[at:at + m].cpu(), wc) and torch.equal(scales[at:at + m].cpu(), ws)
    # every row: off by half a step of its own at most (2^-4), zeros as zeros
    for at in range(0, rows, 1 << 20):
        v, w = src[at:min(at + (1 << 20), rows)].float(), out[at:min(at + (1 << 20), rows)].float()
        e = torch.exp2(scales[at:min(at + (1 << 20), rows)].float() - 127 - 10).repeat_interleave(32, 1)
        assert ((w - v).abs() <= torch.maximum(v.abs() * 2.0 ** -4, e)).all()


def _every_call(b, mats, out, ws, wsb):
    """One pass through each entry point from b.x and b.dy into the tensors of `out`; allocates nothing."""
    T, d, f, t = b.T, b.d, b.f, FT[b.t]
    act = ACT[b.kind]
    ft.ft_gated_ffn(b.x, d, T, d, f, t, act, b.wg, b.wu, b.wd, b.dy, d, out["y"], d, t, out["saved"], ft.FT_SAVE_MX8, ws, wsb)
    ft.ft_act8_pack(b.x, d, T, d, t, out["codes"], out["scales"])
    ft.ft_act8_unpack(out["codes"], out["scales"], T, d, t, out["x"], d)
    ft.ft_gated_ffn_bwd(out["codes"], d, out["scales"], T, d, f, t, act, b.wg, b.wu, b.wd, out["saved"], ft.FT_SAVE_MX8, b.dy,
                        d, out["dx"], d, out["dwg"], out["dwu"], out["dwd"], ws, wsb)
    ft.ft_gated_ffn_bwd(b.x, d, None, T, d, f, t, act, b.wg, b.wu, b.wd, None, ft.FT_SAVE_NONE, b.dy, d, out["dx2"], d, None,
                        None, None, ws, wsb)
    ft.ft_gated_ffn(b.x, d, 5, d, f, t, act, b.wg, b.wu, b.wd, None, d, out["y5"], d, t, None, ft.FT_SAVE_NONE, ws, wsb)
    ft.ft_w4_gated_ffn(b.x, d, T, t, act, *(m[1] for m in mats), None, d, out["w4"], d, t, ws, wsb)
    ft.ft_w4_gemv(b.x, d, 7, t, mats[0][1], None, f, out["g4"], f, FT["fp32"])


def _setup(T, d, f, seed):
    torch = torch_mod()
    from tests.test_gpu_w4_exact import _ints, _pack
    b = Block(T, d, f, "bf16", "silu", seed=seed)
    mats = [_pack(_ints(b.g, -8, 7, n, k), None, torch.rand(n, k // 64, generator=b.g) * 0.01 + 0.002, 64, "bf16")
            for n, k in ((f, d), (f, d), (d, f))]
    wsb = max(ft.ft_gated_ffn_workspace_bytes(T, d, f), ft.ft_w4_gated_ffn_workspace_bytes(T, f),
              *(ft.ft_gated_ffn_bwd_workspace_bytes(T, d, f, s, True) for s in SAVE.values()))
    return b, mats, wsb


def _outputs(b):
    torch = torch_mod()
    T, d, f, dt = b.T, b.d, b.f, b.dt
    e = lambda *s, dtype=dt: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    u8 = torch.uint8
    return dict(y=e(T, d), saved=e(ft.ft_gated_ffn_saved_bytes(T, f, ft.FT_SAVE_MX8), dtype=u8), codes=e(T, d, dtype=u8),
                scales=e(T, d // 32, dtype=u8), x=e(T, d), dx=e(T, d), dwg=e(f, d), dwu=e(f, d), dwd=e(d, f), dx2=e(T, d),
                y5=e(5, d), w4=e(T, d), g4=e(7, f, dtype=torch.float32))


def test_captured_with_shared_tiles():
    """Every entry point in one graph, on tiles that several blocks share, replayed with other inputs between eager calls
    in a workspace of their own."""
    torch = torch_mod()
    b, mats, wsb = _setup(300, 2048, 1024, 25)
    ws, ws_eager = (torch.empty(wsb, dtype=torch.uint8, device="cuda") for _ in range(2))
    out, want = _outputs(b), _outputs(b)
    _every_call(b, mats, out, ws, wsb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _every_call(b, mats, out, ws, wsb)
    for i in range(4):
        b.x.copy_(b.rnd(b.T, b.d))
        b.dy.copy_(b.rnd(b.T, b.d, std=0.3))
        _every_call(b, mats, want, ws_eager, wsb)
        torch.cuda.synchronize()
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[k]), (i, k)


def test_two_calls_at_once():
    """Two streams with a workspace and outputs each, the same weights and inputs: the bits of one call alone."""
    torch = torch_mod()
    b, mats, wsb = _setup(300, 2048, 1024, 26)
    want = _outputs(b)
    ws = [torch.empty(wsb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [_outputs(b) for _ in range(2)]
    _every_call(b, mats, want, ws[0], wsb)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, o, w in zip(streams, outs, ws):
            with torch.cuda.stream(s):
                _every_call(b, mats, o, w, wsb)
    torch.cuda.synchronize()
    for o in outs:
        for k in o:
            assert torch.equal(o[k], want[k]), k


def test_rows_alone_and_in_a_batch():
    """A row's y, dx and 4-bit product have the same bits whatever rows stand beside it, within one form (the same
    number of rows): a padded batch's padding does not reach the others."""
    torch = torch_mod()
    for T in (7, 40, 300):
        _say("padding", T)
        b, mats, wsb = _setup(T, 512, 256, 27)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        outs = []
        for pad in (0.0, float("nan"), 3e4):
            o = _outputs(b)
            b.x[T - 2:] = pad
            b.dy[T - 2:] = pad
            _every_call(b, mats, o, ws, wsb)
            torch.cuda.synchronize()
            outs.append({k: o[k][:T - 2] for k in ("y", "dx", "dx2", "x", "codes", "scales", "w4")})
        for o in outs[1:]:
            for k in o:
                assert torch.equal(o[k], outs[0][k]), (T, k)
