"""GPU tests of the routed layer with 8-bit records where h's codes change hands: made by each block of the down product for
itself (rows of h up to 4096 elements, 24576 in all) or by a launch of their own."""
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_moe_layer import Layer, _dt, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,f,E,k", [
    (1, 256, 4096, 3, 2), (1, 256, 4112, 3, 2), (2, 64, 4096, 8, 3), (1, 64, 24576, 2, 1), (1, 64, 3056, 9, 8), (3, 48, 1024, 12, 8),
    (5, 48, 1024, 12, 5),
])
def test_codes_of_h(T, d, f, E, k):
    torch = torch_mod()
    _say("moe codes", T, d, f, E, k)
    L = Layer(T, d, f, E, k, "i8", 71)
    b = L.buffers("fp32")
    r = torch.randn(T, d, generator=L.g).to(_dt("fp32")).cuda()
    L.call(b, "fp32", r)
    L.check(b, "fp32", r)
