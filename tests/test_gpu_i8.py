"""GPU tests of the products in 8-bit integers against plain forms in 64 bits, through the C ABI.

Codes, scales and whole-number sums are compared for equality; blocks within the elementwise bounds
of tests/i8_ref.py.
"""
import pytest

from moe_expert_offload_amd import ft
from tests import dense_ref as R
from tests import i8_ref as I8
from tests.gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu

FT = {"bf16": ft.FT_T_BF16, "fp16": ft.FT_T_FP16, "fp32": ft.FT_T_FP32}
ACT = {"silu": ft.FT_ACT_SILU, "gelu": ft.FT_ACT_GELU_TANH}


def _say(*a):
    print("[case]", *a, flush=True)


def _dt(t):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[t]


def _gen(*key):
    torch = torch_mod()
    s = 17
    for k in key:
        s = (s * 1000003 + int(k)) % (1 << 31)
    return torch.Generator().manual_seed(s)


def _quant(x, t, ld=None, rows=None, n=None, stream=None):
    torch = torch_mod()
    rows, n = rows or x.shape[0], n or x.shape[1]
    codes = torch.full((rows, n), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), 7.0, device="cuda")
    ft.ft_i8_quant(x, ld or n, rows, n, FT[t], codes, scales, stream)
    return codes, scales


def _same_scales(got, want):
    torch = torch_mod()
    g = got.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(g, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


@pytest.mark.parametrize("rows,n,t", [
    (1, 16, "bf16"), (3, 16, "fp16"), (5, 48, "bf16"), (7, 1024, "fp16"), (9, 1040, "bf16"), (257, 2048, "fp16"),
    (33, 4096, "bf16"), (6, 4112, "fp16"), (1, 11008, "bf16"), (2, 65536, "fp16"), (5000, 112, "bf16"), (1031, 528, "fp16"),
    (2100, 4096, "bf16"),
])
def test_quant(rows, n, t):
    torch = torch_mod()
    _say("quant", rows, n, t)
    g = _gen(rows, n)
    x = torch.randn(rows, n, generator=g).to(_dt(t))
    x[0, -1] = 127 / 8  # a scale of a power of two: halves are ties
    x[0, :8] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 62.5, 126.5, -3.5]) / 8
    x[rows // 2, :] *= 0 if rows > 2 else 1
    if rows > 4:
        x[1] *= 2.0 ** -13 if t == "fp16" else 2.0 ** -125  # subnormal elements
        x[3, n - 3] = float("inf")
        x[4, 2] = float("nan")
    codes, scales = _quant(x.cuda(), t)
    torch.cuda.synchronize()
    q, s = I8.quant(x)
    assert torch.equal(codes.cpu(), q)
    _same_scales(scales, s)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_quant_every_value(t):
    """Every finite 16-bit pattern, under largest elements of many kinds."""
    torch = torch_mod()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(_dt(t))
    v = v[torch.isfinite(v.float())]
    tops = [1.0, 127.0, 0.0625 * 127, 1.9921875, 0.335, 3.3895e38 if t == "bf16" else 65504.0, 1e-3,
            2.0 ** -133 if t == "bf16" else 2.0 ** -24, 3 * 2.0 ** -130 if t == "bf16" else 5 * 2.0 ** -24, 1e-37 if t == "bf16" else 6e-5]
    rows = []
    for top in tops:
        top = torch.tensor(top).to(_dt(t))
        r = torch.where(v.double().abs() <= top.double(), v, torch.zeros((), dtype=v.dtype))
        r = torch.cat([top.reshape(1), r])
        rows.append(torch.nn.functional.pad(r.view(torch.int16), (0, 65536 - r.numel())).view(_dt(t)))
    x = torch.stack(rows)
    _say("quant every value", t, tuple(x.shape))
    codes, scales = _quant(x.cuda(), t)
    torch.cuda.synchronize()
    q, s = I8.quant(x)
    assert torch.equal(codes.cpu(), q)
    _same_scales(scales, s)


@pytest.mark.parametrize("rows,n,ld,t", [(5, 48, 64, "bf16"), (300, 1056, 1064, "fp16")])
def test_quant_strides(rows, n, ld, t):
    torch = torch_mod()
    _say("quant strides", rows, n, ld)
    x = torch.randn(rows, ld, generator=_gen(rows, ld)).to(_dt(t))
    x[:, n:] = float("nan")  # padding is not read
    codes, scales = _quant(x.cuda(), t, ld, rows, n)
    torch.cuda.synchronize()
    q, s = I8.quant(x[:, :n])
    assert torch.equal(codes.cpu(), q)
    _same_scales(scales, s)


def _weights(g, N, K, std=None):
    torch = torch_mod()
    codes = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    scales = (torch.rand(N, generator=g) + 0.5) * ((std or K ** -0.5) / 73.9)
    return codes.cuda(), scales.cuda()


def _gemm(x, xs, w, t, T, N, K, y_t, res=None, ldx=None, ldr=None, y=None, ldy=None, wsb=None, stream=None):
    torch = torch_mod()
    if y is None:
        y = torch.full((T, N), 7.0, dtype=_dt(y_t), device="cuda")
    wsb = wsb or ft.ft_i8_gemm_workspace_bytes(T, N, K, xs is not None)
    ws = torch.full((wsb,), 0x5a, dtype=torch.uint8, device="cuda")
    ft.ft_i8_gemm(x, ldx or K, xs, T, FT[t], ft.make_i8_matrix(w[0], w[1], N, K), res, ldr or N, y, ldy or N, FT[y_t], ws,
                  wsb, stream)
    return y, ws


def _want_f32(q, s, w):
    """fp32 bits of the product: the whole-number sum rounded once, then two products."""
    torch = torch_mod()
    acc = (q.cuda().double() @ w[0].double().t()).float()
    return (acc * w[1].float()) * s.cuda().float()[:, None]


SIZES = [
    (1, 1, 16), (1, 17, 48), (1, 4096, 4096), (2, 4099, 1040), (15, 24, 65536), (16, 130, 272), (17, 129, 2048), (31, 1000, 304),
    (33, 77, 512), (64, 520, 1104), (65, 33, 160), (66, 300, 1040), (127, 136, 208), (128, 128, 128), (129, 1001, 272), (200, 4096, 528),
    (300, 1055, 4096), (513, 257, 144), (700, 2050, 1040), (1021, 5632, 2048), (2053, 4104, 1296), (4100, 1056, 144),
]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_gemm_bits(T, N, K):
    """fp32 results without a residual: equal bits, codes in hand."""
    torch = torch_mod()
    _say("gemm bits", T, N, K)
    g = _gen(T, N, K)
    x = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8).cuda()
    xs = ((torch.rand(T, generator=g) + 0.5) * 0.02).cuda()
    w = _weights(g, N, K)
    y, _ = _gemm(x, xs, w, "bf16", T, N, K, "fp32")
    torch.cuda.synchronize()
    assert torch.equal(y, _want_f32(x, xs, w))


@pytest.mark.parametrize("T,N,K,t,y_t,res", [
    (1, 40, 64, "bf16", "bf16", True), (1, 4099, 11008, "fp16", "fp16", False), (5, 1000, 272, "fp16", "fp32", True),
    (13, 513, 2048, "bf16", "bf16", True), (40, 72, 160, "bf16", "fp32", True), (64, 264, 96, "fp16", "fp16", True),
    (100, 77, 336, "bf16", "bf16", True), (260, 1032, 144, "fp16", "fp16", True), (1030, 515, 400, "bf16", "fp32", True),
    (2050, 2056, 272, "fp16", "fp16", False),
])
def test_gemm(T, N, K, t, y_t, res):
    torch = torch_mod()
    _say("gemm", T, N, K, t, y_t, res)
    g = _gen(T, N, K)
    x = torch.randn(T, K, generator=g).to(_dt(t)).cuda()
    w = _weights(g, N, K)
    r = torch.randn(T, N, generator=g).to(_dt(y_t)).cuda() if res else None
    y, _ = _gemm(x, None, w, t, T, N, K, y_t, r)
    torch.cuda.synchronize()
    want = I8.product(*I8.quant(x), *w)
    if res:
        want = R.add(want, R.exactly(r))
    R.check(y, R.rounded(want, _dt(y_t)), "y")


@pytest.mark.parametrize("T,N,K", [(3, 33, 64), (90, 136, 176), (600, 250, 272), (4096, 4096, 256)])
def test_gemm_strides(T, N, K):
    """Row strides of every operand, in place residual, unaligned y; nothing outside the result is written."""
    torch = torch_mod()
    _say("gemm strides", T, N, K)
    g = _gen(T, N, K, 3)
    x = torch.full((T, K + 24), float("nan")).to(torch.bfloat16)
    x[:, :K] = torch.randn(T, K, generator=g)
    w = _weights(g, N, K)
    for ldy, off, y_t in ((N + 5, 3, "bf16"), (N + 8, 8, "fp32"), (N, 0, "bf16")):
        flat = torch.full((T * ldy + 16,), 5.0, dtype=_dt(y_t), device="cuda")
        y = flat[off:off + T * ldy].view(T, ldy)
        r = torch.randn(T, N, generator=g).to(_dt(y_t)).cuda()
        y[:, :N] = r
        _gemm(x.cuda(), None, w, "bf16", T, N, K, y_t, y, K + 24, ldy, y, ldy)
        torch.cuda.synchronize()
        want = R.rounded(R.add(I8.product(*I8.quant(x[:, :K]), *w), R.exactly(r)), _dt(y_t))
        R.check(y[:, :N], want, "y")
        left = flat.clone()
        left[off:off + T * ldy].view(T, ldy)[:, :N] = 5.0
        assert (left == 5.0).all()


@pytest.mark.parametrize("T", [4, 70, 300])
def test_rows_not_finite(T):
    """Rows that are not finite become NaN, their neighbours do not."""
    torch = torch_mod()
    N, K = 72, 160
    _say("gemm not finite", T)
    g = _gen(T)
    x = torch.randn(T, K, generator=g).to(torch.float16)
    x[1, 7], x[T - 1, K - 1] = float("nan"), float("-inf")
    w = _weights(g, N, K)
    y, _ = _gemm(x.cuda(), None, w, "fp16", T, N, K, "fp32")
    torch.cuda.synchronize()
    bad = torch.zeros(T, dtype=torch.bool)
    bad[1] = bad[T - 1] = True
    assert torch.isnan(y.cpu()[bad]).all() and torch.isfinite(y.cpu()[~bad]).all()
    q, s = I8.quant(x[~bad])
    assert torch.equal(y[~bad.cuda()], _want_f32(q, s, w))


def _ffn(x, w, t, kind, T, d, f, y_t, res=None, ldx=None, ldy=None, y=None, ldr=None, stream=None):
    torch = torch_mod()
    if y is None:
        y = torch.full((T, d), 7.0, dtype=_dt(y_t), device="cuda")
    wsb = ft.ft_i8_gated_ffn_workspace_bytes(T, d, f)
    ws = torch.full((wsb,), 0x5a, dtype=torch.uint8, device="cuda")
    m = [ft.make_i8_matrix(*w[0], f, d), ft.make_i8_matrix(*w[1], f, d), ft.make_i8_matrix(*w[2], d, f)]
    ft.ft_i8_gated_ffn(x, ldx or d, T, FT[t], ACT[kind], *m, res, ldr or d, y, ldy or d, FT[y_t], ws, wsb, stream)
    return y, ws


FFN = [
    (1, 16, 16, "bf16", "silu", "bf16", False), (1, 2048, 768, "fp16", "silu", "fp32", True), (1, 4096, 1104, "bf16", "gelu", "bf16", False),
    (5, 272, 96, "bf16", "silu", "fp32", True), (16, 512, 1040, "fp16", "gelu", "fp16", True), (17, 96, 400, "bf16", "silu", "bf16", False),
    (33, 160, 144, "fp16", "silu", "fp16", False), (64, 112, 528, "bf16", "silu", "fp32", True), (65, 528, 112, "bf16", "gelu", "bf16", True),
    (130, 208, 304, "fp16", "silu", "fp32", False), (300, 272, 784, "bf16", "silu", "bf16", True), (1030, 400, 2064, "fp16", "silu", "fp16", True),
    (2100, 1040, 272, "bf16", "gelu", "bf16", False),
]


@pytest.mark.parametrize("T,d,f,t,kind,y_t,res", FFN)
def test_ffn(T, d, f, t, kind, y_t, res):
    torch = torch_mod()
    _say("ffn", T, d, f, t, kind, y_t, res)
    g = _gen(T, d, f)
    x = torch.randn(T, d, generator=g).to(_dt(t)).cuda()
    w = _weights(g, f, d), _weights(g, f, d), _weights(g, d, f)
    r = torch.randn(T, d, generator=g).to(_dt(y_t)).cuda() if res else None
    y, _ = _ffn(x, w, t, kind, T, d, f, y_t, r)
    torch.cuda.synchronize()
    want = I8.ffn(x, *w, kind, _dt(t), R.exactly(r) if res else None, _dt(y_t))
    R.check(y, want, "y")


@pytest.mark.parametrize("T,d,f", [(1, 256, 512), (40, 512, 256), (300, 512, 1040), (4200, 272, 512)])
def test_ffn_whole_numbers(T, d, f):
    """Gates of 64 and more are their own SiLU: h is u's multiple, a whole number, and y's bits follow from it."""
    torch = torch_mod()
    _say("ffn whole numbers", T, d, f)
    g = _gen(T, d, f, 9)
    x = torch.zeros(T, d)
    x[:, 0] = 127  # the row's scale is 1
    x[:, 1:4] = torch.randint(-4, 5, (T, 3), generator=g).float()
    gate = torch.zeros(f, d, dtype=torch.int8)
    gate[:, 0] = 1  # a = 127
    up = torch.randint(-1, 2, (f, d), generator=g, dtype=torch.int8)
    up[:, 0] = 0
    up[0, :4] = torch.tensor([1, 0, 0, 0])  # u = 127, h = 127 * 127 / 128: the row's largest
    down = torch.randint(-128, 128, (d, f), generator=g, dtype=torch.int8)
    one = torch.ones(f)
    us = torch.full((f,), 2.0 ** -4)
    us[0] = 2.0 ** -3
    ds = torch.rand(d, generator=g) + 0.5
    w = [(gate.cuda(), one.cuda()), (up.cuda(), us.cuda()), (down.cuda(), ds.cuda())]
    y, _ = _ffn(x.to(torch.bfloat16).cuda(), w, "bf16", "silu", T, d, f, "fp32")
    torch.cuda.synchronize()
    h = (127.0 * (x @ up.float().t() * us)).to(torch.bfloat16)
    q, s = I8.quant(h)
    assert torch.equal(y, _want_f32(q, s, w[2]))


def test_ffn_strides_and_composition():
    """The block equals its parts called one after the other, rows strided."""
    torch = torch_mod()
    for T in (3, 80):
        d, f = 272, 400
        g = _gen(T, 5)
        x = torch.full((T, d + 8), float("nan"), dtype=torch.float16)
        x[:, :d] = torch.randn(T, d, generator=g)
        x = x.cuda()
        w = _weights(g, f, d), _weights(g, f, d), _weights(g, d, f)
        y = torch.full((T, d + 3), 7.0, dtype=torch.float16, device="cuda")
        _ffn(x, w, "fp16", "silu", T, d, f, "fp16", None, d + 8, d + 3, y)
        torch.cuda.synchronize()
        want = I8.ffn(x[:, :d], *w, "silu", torch.float16, None)
        R.check(y[:, :d], want, "y")
        assert (y[:, d:] == 7.0).all()


def test_offsets_past_32_bits():
    """A result of more than 2^31 elements and weights of more than 2^31 bytes."""
    torch = torch_mod()
    _say("large")
    T, N, K = 5, 34 * 1024 * 1024 + 5, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.rand(N, generator=g, device="cuda")
    x = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.ones(T, device="cuda")
    y, _ = _gemm(x, xs, (codes, scales), "bf16", T, N, K, "fp32")
    torch.cuda.synchronize()
    sl = slice(N - 3000, N)
    assert torch.equal(y[:, sl], _want_f32(x, xs, (codes[sl], scales[sl])))
    del y, codes, scales
    T, N, K = 2 ** 22 + 3, 515, 48
    x = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(T, generator=g, device="cuda")
    w = _weights(_gen(4), N, K)
    y, _ = _gemm(x, xs, w, "bf16", T, N, K, "fp32")
    torch.cuda.synchronize()
    for sl in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        assert torch.equal(y[sl], _want_f32(x[sl], xs[sl], w))


@pytest.mark.parametrize("T", [1, 20, 70, 300, 1024])
def test_captured_and_equal_bits(T):
    """Every entry point captured, replayed between eager work on changed inputs, equal to eager calls."""
    torch = torch_mod()
    d, f = 528, 784
    _say("graph", T)
    g = _gen(T, 8)
    w = _weights(g, f, d), _weights(g, f, d), _weights(g, d, f)
    xs_ = [torch.randn(T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    x = xs_[0].clone()
    y = torch.empty(T, d, device="cuda")
    z = torch.empty(T, f, dtype=torch.bfloat16, device="cuda")
    ws1 = torch.empty(ft.ft_i8_gated_ffn_workspace_bytes(T, d, f), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(ft.ft_i8_gemm_workspace_bytes(T, f, d, 0), dtype=torch.uint8, device="cuda")
    m = [ft.make_i8_matrix(*w[0], f, d), ft.make_i8_matrix(*w[1], f, d), ft.make_i8_matrix(*w[2], d, f)]

    def calls():
        ft.ft_i8_gated_ffn(x, d, T, FT["bf16"], ACT["silu"], *m, None, d, y, d, FT["fp32"], ws1, ws1.numel())
        ft.ft_i8_gemm(x, d, None, T, FT["bf16"], m[0], None, f, z, f, FT["bf16"], ws2, ws2.numel())

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for v in xs_:
        x.copy_(v)
        calls()
        torch.cuda.synchronize()
        want = y.clone(), z.clone()
        y.zero_()
        z.zero_()
        ws1.fill_(0xee)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own."""
    torch = torch_mod()
    _say("two streams")
    T, d, f = 300, 1040, 2064
    g = _gen(77)
    w = _weights(g, f, d), _weights(g, f, d), _weights(g, d, f)
    x = [torch.randn(T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [_ffn(v, w, "bf16", "silu", T, d, f, "bf16")[0] for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(v) for v in want]
    wss = [torch.empty(ft.ft_i8_gated_ffn_workspace_bytes(T, d, f), dtype=torch.uint8, device="cuda") for _ in range(2)]
    m = [ft.make_i8_matrix(*w[0], f, d), ft.make_i8_matrix(*w[1], f, d), ft.make_i8_matrix(*w[2], d, f)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            ft.ft_i8_gated_ffn(x[i], d, T, FT["bf16"], ACT["silu"], *m, None, d, outs[i], d, FT["bf16"], wss[i], wss[i].numel(),
                               streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
