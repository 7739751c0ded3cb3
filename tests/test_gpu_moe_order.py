"""GPU tests of the routed layer's order of sums: it goes by the shape and the number of tokens alone, so a token's row
has the same bits whatever the other tokens are, whatever experts they take and whichever of those have a record."""
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_moe_layer import Layer, _say

pytestmark = pytest.mark.gpu

# T, d, f, E, k: the matrix form, on rows of y that blocks share (d up to 2048) and that they do not; the row form
SHAPES = [
    (64, 2048, 128, 16, 8),
    (64, 1024, 256, 12, 5),
    (40, 512, 384, 6, 4),
    (48, 768, 128, 9, 8),
    (64, 256, 128, 3, 3),  # fewer experts than blocks that share rows
    (33, 2304, 128, 4, 4),
    (9, 1024, 128, 64, 8),
]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
@pytest.mark.parametrize("T,d,f,E,k", SHAPES)
def test_rows_do_not_hang_on_others(T, d, f, E, k, fmt):
    torch = torch_mod()
    _say("moe order", T, d, f, E, k, fmt)
    L = Layer(T, d, f, E, k, fmt, 31)
    kept = [0, T // 2, T - 1]
    others = [t for t in range(T) if t not in kept]
    b = L.buffers("fp32")
    L.call(b, "fp32")
    L.check(b, "fp32")
    want, idx = b["y"][kept].clone(), b["idx"][kept].clone()
    for turn in range(8):
        L.x[others] = torch.randn(len(others), d, generator=L.g).to(torch.bfloat16)
        m = torch.ones(T, E, dtype=torch.uint8)
        for t in others:  # other experts for the others, more and fewer of them
            m[t, torch.randperm(E, generator=L.g)[:turn % E]] = 0
        L.allowed = m.cuda()
        L.dx.copy_(L.x)
        L.call(b, "fp32")
        torch.cuda.synchronize()
        assert torch.equal(b["idx"][kept], idx)
        assert torch.equal(b["y"][kept], want), turn
    L.check(b, "fp32")


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
@pytest.mark.parametrize("T,d,f,E,k", [(64, 2048, 128, 24, 4), (64, 512, 128, 12, 3), (16, 1024, 128, 64, 8)])
def test_rows_do_not_hang_on_absent_experts(T, d, f, E, k, fmt):
    """Experts that a row does not take lose their records, one after the other."""
    torch = torch_mod()
    _say("moe order, absent experts", T, d, f, E, k, fmt)
    L = Layer(T, d, f, E, k, fmt, 37)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    torch.cuda.synchronize()
    row = T // 3
    want = b["y"][row].clone()
    free = sorted(set(range(E)) - set(b["idx"][row].tolist()))
    slots = torch.arange(E, dtype=torch.int32)
    for e in free:
        slots[e] = -1
        L.slot_of = slots.cuda()
        L.call(b, "fp32")
        torch.cuda.synchronize()
        assert torch.equal(b["y"][row], want), e
    L.check(b, "fp32")
