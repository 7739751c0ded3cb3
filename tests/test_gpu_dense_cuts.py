"""GPU tests of the dense block over every way its tiled products are cut (which case reaches which:
test_dense_cut.py), on whole-number inputs whose sums are exact in fp32: every output is compared for equality."""
import pytest

from moe_expert_offload_amd import ft
from tests import dense_cuts as C
from tests.gpu_helpers import torch_mod
from tests.test_gpu_dense import ACT, FT, SAVE, _dt, _say

pytestmark = pytest.mark.gpu


def _same(got, want, what):
    torch = torch_mod()
    wrong = got != want
    n = int(wrong.sum())
    if n:
        at = torch.nonzero(wrong)
        print(f"[wrong] {what}: {n} of {wrong.numel()}, rows {at[:, 0].min().item()} .. {at[:, 0].max().item()}, columns "
              f"{at[:, 1].min().item()} .. {at[:, 1].max().item()}", flush=True)
    assert n == 0 and torch.isfinite(got.float()).all(), (what, n)


def _workspace(n):
    torch = torch_mod()
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # NaN in every format: a slot read but not written would show
    return ws


@pytest.mark.parametrize("T,d,f,t,kind,save,res,y_t,ways", C.FORWARD)
def test_forward_exact(T, d, f, t, kind, save, res, y_t, ways):
    torch = torch_mod()
    _say("ffn exact", T, d, f, t, kind, save, res, y_t, ways)
    w = C.Whole(T * 31 + d * 7 + f, "cuda")
    dt, yt = _dt(t), _dt(y_t)
    x, wg, wu, wd = w.weights(T, d, f)
    r = w.numbers(-200, 200, T, d) if res else None
    a, u, h, y = C.forward(x, wg, wu, wd, dt, r)
    assert C.gates_ok(a) and u.abs().max() <= 256 and C.exact_in_fp32(h, wd.t())
    gx, gg, gu, gd = (v.to(dt) for v in (x, wg, wu, wd))
    got = torch.full((T, d), 7.0, dtype=yt, device="cuda")
    n = ft.ft_gated_ffn_saved_bytes(T, f, SAVE[save])
    saved = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    wsb = ft.ft_gated_ffn_workspace_bytes(T, d, f)
    ft.ft_gated_ffn(gx, d, T, d, f, FT[t], ACT[kind], gg, gu, gd, None if r is None else r.to(yt), d, got, d, FT[y_t], saved,
                    SAVE[save], _workspace(wsb), wsb)
    torch.cuda.synchronize()
    if save == "16":
        for i, (v, k) in enumerate(((a, "a"), (u, "u"))):
            _same(saved[2 * T * f * i:2 * T * f * (i + 1)].view(dt).reshape(T, f), v.to(dt), k)
    if save == "mx8":
        for i, (v, k) in enumerate(((a, "a"), (u, "u"))):
            codes, scales = C.mx8(v)
            # (the sign of a zero is the sum's own)
            here = saved[T * f * i:T * f * (i + 1)].reshape(T, f)
            _same(torch.where(here == 128, 0, here), torch.where(codes == 128, 0, codes), k + " codes")
            m = T * (f // 32)
            _same(saved[2 * T * f + m * i:2 * T * f + m * (i + 1)].reshape(T, f // 32), scales, k + " scales")
    _same(got, C.rounded(y, yt), "y")


@pytest.mark.parametrize("T,d,f,t,kind,save,x8,ways", C.BACKWARD)
def test_backward_exact(T, d, f, t, kind, save, x8, ways):
    torch = torch_mod()
    _say("bwd exact", T, d, f, t, kind, save, x8, ways)
    w = C.Whole(T * 13 + d * 5 + f, "cuda")
    dt = _dt(t)
    x, wg, wu, wd = w.weights(T, d, f)
    dy = w.gradient(T, d) * (2.0 ** -8 if t == "fp16" else 1.0)  # keeps fp16's sums below its end
    unit = 2.0 ** -8 if t == "fp16" else 1.0
    gx, xs, saved = x.to(dt), None, None
    if x8:
        gx = x.float().to(torch.float8_e4m3fn).view(torch.uint8)
        xs = w.numbers(127, 128, T, d // 32).to(torch.uint8)
        x = C.mx8_values(gx, xs)
    if save == "none":
        a, u = x @ wg.t(), x @ wu.t()
    elif save == "16":
        a, u = w.kept(T, f)
        saved = torch.cat([v.to(dt).view(torch.uint8).flatten() for v in (a, u)])
    else:
        (ac, asc), (uc, usc) = w.kept_mx8(T, f)
        a, u = C.mx8_values(ac, asc), C.mx8_values(uc, usc)
        saved = torch.cat([v.flatten() for v in (ac, uc, asc, usc)])
    assert a.min() >= 33
    want = C.backward(x, wg, wu, wd, a, u, dy, dt)
    assert C.exact_in_fp32(dy / unit, wd)
    assert C.exact_in_fp32(torch.cat([want["da"], want["du"]], 1) / unit, torch.cat([wg, wu]))
    for p, q in ((want["da"].t() / unit, x), (want["du"].t() / unit, x), (dy.t() / unit, want["h"])):
        assert C.exact_in_fp32(p, q)
    out = [torch.full(s, 7.0, dtype=dt, device="cuda") for s in ((T, d), (f, d), (f, d), (d, f))]
    wsb = ft.ft_gated_ffn_bwd_workspace_bytes(T, d, f, SAVE[save], x8)
    ft.ft_gated_ffn_bwd(gx, d, xs, T, d, f, FT[t], ACT[kind], *(v.to(dt) for v in (wg, wu, wd)), saved, SAVE[save],
                        dy.to(dt), d, out[0], d, *out[1:], _workspace(wsb), wsb)
    torch.cuda.synchronize()
    for g, k in zip(out, ("dx", "dwg", "dwu", "dwd")):
        _same(g, C.rounded(want[k], dt), k)
