"""Products in 8-bit integers by every way of cutting, on whole numbers: equal bits (GPU)."""
import pytest

from tests import i8_cuts as C
from tests import i8_ref as I8
from tests.gpu_helpers import torch_mod
from tests.test_gpu_i8 import _ffn, _gemm, _gen, _say, _want_f32, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,way", C.GEMM)
def test_product(T, N, K, way):
    torch = torch_mod()
    _say("product", T, N, K, way)
    g = _gen(T, N, K, 1)
    x = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8).cuda()
    xs = ((torch.rand(T, generator=g) + 0.5) * 0.02).cuda()
    w = _weights(g, N, K)
    y, _ = _gemm(x, xs, w, "bf16", T, N, K, "fp32")
    z, _ = _gemm(x, xs, w, "fp16", T, N, K, "fp16")
    torch.cuda.synchronize()
    want = _want_f32(x, xs, w)
    assert torch.equal(y, want)
    assert torch.equal(z, want.half())


@pytest.mark.parametrize("T,d,f,up_way,down_way", C.FFN)
def test_block(T, d, f, up_way, down_way):
    """Gates of 127 and more are their own SiLU, so every step has one right value; each k takes part."""
    torch = torch_mod()
    _say("block", T, d, f, up_way, down_way)
    g = _gen(T, d, f, 2)
    x = torch.randint(0, 3, (T, d), generator=g, dtype=torch.int8)
    x[:, 0] = 127  # the rows' scale is 1
    gate = torch.randint(0, 2, (f, d), generator=g, dtype=torch.int8)
    gate[:, 0] = 1  # a >= 127
    up = torch.randint(-2, 3, (f, d), generator=g, dtype=torch.int8)
    down = torch.randint(-128, 128, (d, f), generator=g, dtype=torch.int8)
    one = torch.ones(f)
    us, ds = torch.full((f,), 2.0 ** -4), torch.rand(d, generator=g) + 0.5
    us[f // 2:] = 2.0 ** -6
    x, w = x.cuda(), [(gate.cuda(), one.cuda()), (up.cuda(), us.cuda()), (down.cuda(), ds.cuda())]
    y, _ = _ffn(x.to(torch.bfloat16), w, "bf16", "silu", T, d, f, "fp32")
    torch.cuda.synchronize()
    a, u = ((x.double() @ m[0].double().t()).float() * m[1] for m in w[:2])
    q, s = I8.quant((a * u).to(torch.bfloat16))
    assert torch.equal(y, _want_f32(q, s, w[2]))
