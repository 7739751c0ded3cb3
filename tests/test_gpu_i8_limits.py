"""GPU tests of the products in 8-bit integers at the largest sum of whole numbers that their sizes allow: -128 times -128 along
2^16 elements, 2^30."""
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_i8 import _gemm, _say, _want_f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 3, 16, 40, 70, 300])
def test_largest_sum(T):
    torch = torch_mod()
    N, K = 136, 65536
    _say("gemm largest sum", T)
    x = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    codes = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    codes[1::3] = 127
    codes[2::3, 1:] = 127
    xs = (torch.arange(T, device="cuda") + 1) * 2.0 ** -20
    scales = (torch.arange(N, device="cuda") + 1) * 2.0 ** -12
    y, _ = _gemm(x, xs, (codes, scales), "bf16", T, N, K, "fp32")
    torch.cuda.synchronize()
    assert torch.equal(y, _want_f32(x, xs, (codes, scales)))
    # 2^30 exactly, and two powers of two beside it
    assert y[0, 0].item() == 2.0 ** (30 - 20 - 12)
