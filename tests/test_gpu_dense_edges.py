"""GPU tests of the dense operators' contracts at their edges, through the C ABI."""
import pytest

from moe_expert_offload_amd import ft
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
