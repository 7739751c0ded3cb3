"""GPU tests of the routed layer for a few tokens against a plain form in 64 bits, through the C ABI.

Experts and gates are the router's, bit for bit; y is within the elementwise bounds of
tests/moe_ref.py for those."""
import pytest

from moe_expert_offload_amd import ft
from tests import dense_ref as R
from tests import moe_ref as M
from tests.gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu

FMT = {"bf16": ft.FT_W_BF16, "mxfp4": ft.FT_W_MXFP4, "i8": ft.FT_W_I8}
FT = {"bf16": ft.FT_T_BF16, "fp32": ft.FT_T_FP32}


def _say(*a):
    print("[case]", *a, flush=True)


def _dt(t):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[t]


class Layer:
    def __init__(self, T, d, f, E, k, fmt, seed=0, n_slots=None):
        torch = torch_mod()
        self.T, self.d, self.f, self.E, self.k, self.fmt = T, d, f, E, k, fmt
        self.g = g = torch.Generator().manual_seed(seed * 7919 + T * 104729 + d * 31 + f * 17 + E * 5 + k)
        self.x = torch.randn(T, d, generator=g).to(torch.bfloat16)
        self.wr = (torch.randn(E, d, generator=g) * d ** -0.5).to(torch.bfloat16)
        self.n_slots = E if n_slots is None else n_slots
        self.recs = M.records(g, self.n_slots, d, f, fmt)
        self.shape = ft.make_shape(1, E, d, f, k, FMT[fmt])
        assert ft.ft_record_bytes(self.shape) == self.recs.shape[1]
        self.dx, self.dwr, self.drecs = self.x.cuda(), self.wr.cuda(), self.recs.cuda()
        self.slot_of = self.allowed = None

    def buffers(self, y_t, T=None):
        torch = torch_mod()
        T = self.T if T is None else T
        wsb = ft.ft_moe_layer_workspace_bytes(self.shape, T)
        return dict(y=torch.full((T, self.d), 7.0, dtype=_dt(y_t), device="cuda"),
                    idx=torch.full((T, self.k), -9, dtype=torch.int32, device="cuda"),
                    gates=torch.full((T, self.k), 9.0, device="cuda"),
                    ws=torch.full((wsb,), 0xa5, dtype=torch.uint8, device="cuda"))

    def call(self, b, y_t, res=None, T=None, stream=None):
        ft.ft_moe_layer(self.shape, self.dx, self.T if T is None else T, self.dwr, self.allowed, self.drecs, self.n_slots,
                        self.slot_of, res, b["y"], FT[y_t], b["idx"], b["gates"], b["ws"], b["ws"].numel(), stream)

    def routed(self):
        torch = torch_mod()
        idx = torch.empty(self.T, self.k, dtype=torch.int32, device="cuda")
        gates = torch.empty(self.T, self.k, device="cuda")
        logits = torch.empty(self.T, self.E, device="cuda")
        ft.ft_router_topk(self.dx, self.dwr, self.allowed, self.T, self.d, self.E, self.k, idx, gates, logits)
        return idx, gates

    def slots(self):
        if self.slot_of is None:
            return {e: e for e in range(self.E)}
        s = self.slot_of.cpu().tolist()
        return {e: s[e] for e in range(self.E) if 0 <= s[e] < self.n_slots}

    def check(self, b, y_t, res=None, T=None):
        torch = torch_mod()
        torch.cuda.synchronize()
        T = self.T if T is None else T
        idx, gates = (v[:T] for v in self.routed())
        assert torch.equal(b["idx"], idx)
        assert torch.equal(b["gates"], gates)
        want = M.layer(self.x[:T], self.recs, self.slots(), idx.cpu(), gates.cpu(), self.d, self.f, self.fmt, _dt(y_t), res)
        R.check(b["y"], want, "y")


CASES = [
    # T, d, f, E, k, format, y, residual
    (1, 8, 8, 1, 1, "bf16", "fp32", False),
    (1, 16, 16, 3, 2, "i8", "bf16", True),
    (1, 256, 128, 4, 2, "mxfp4", "fp32", False),
    (1, 2048, 768, 16, 8, "bf16", "fp32", True),
    (1, 2048, 768, 16, 8, "i8", "fp32", False),
    (1, 2048, 768, 16, 8, "mxfp4", "bf16", True),
    (1, 4096, 2048, 8, 6, "bf16", "fp32", False),
    (1, 4104, 520, 8, 6, "bf16", "bf16", False),   # rows past one chunk of pieces
    (2, 4096, 2064, 8, 3, "i8", "fp32", True),
    (3, 8192, 128, 4, 2, "mxfp4", "fp32", False),
    (2, 8200, 40, 5, 2, "bf16", "fp32", True),     # more rows of y than 16 a unit
    (5, 264, 40, 7, 3, "bf16", "bf16", True),
    (7, 272, 1040, 300, 5, "i8", "bf16", False),   # more experts than 256
    (9, 512, 384, 11, 4, "mxfp4", "fp32", True),
    (13, 520, 776, 40, 8, "bf16", "fp32", False),
    (16, 1024, 4112, 6, 2, "i8", "fp32", False),
    (16, 768, 4224, 6, 2, "mxfp4", "fp32", False),
    (33, 136, 72, 5, 5, "bf16", "fp32", True),     # every expert by every token
    (40, 1040, 528, 8, 2, "i8", "bf16", True),
    (64, 256, 256, 9, 8, "mxfp4", "bf16", False),  # the most pairs, groups of more than 50
    (64, 2056, 104, 1000, 8, "bf16", "fp32", False),
    (64, 1024, 160, 64, 8, "i8", "bf16", True),
    (63, 2048, 768, 12, 7, "bf16", "fp32", True),
    (36, 2048, 128, 200, 2, "mxfp4", "fp32", False),  # rows of x that LDS does not hold
    (64, 2304, 32, 300, 2, "i8", "fp32", True),
    (9, 512, 4224, 60, 4, "mxfp4", "fp32", False),    # rows of h that LDS does not hold, past one chunk
    (20, 512, 4112, 100, 2, "i8", "bf16", False),
    (2, 8208, 48, 5, 2, "i8", "fp32", False),
    (17, 512, 128, 1, 1, "mxfp4", "fp32", True),      # one expert: 16 tokens and one more
    (32, 264, 72, 2, 2, "bf16", "fp32", False),       # two whole passes of 16
    (48, 1552, 400, 4, 2, "i8", "fp32", True),
    (64, 8200, 24, 3, 3, "bf16", "bf16", False),      # the matrix form on more rows of y than 16 a unit
    (64, 4096, 384, 6, 5, "mxfp4", "fp32", True),
    (20, 16384, 16, 2, 1, "bf16", "fp32", False),     # the widest: parts of 4 tokens, of 8
    (24, 16384, 128, 2, 1, "mxfp4", "bf16", True),
    (30, 16384, 32, 2, 2, "i8", "fp32", False),
    (40, 8, 8, 2, 1, "bf16", "fp32", True),           # the narrowest: 16 blocks share the rows of y
    (37, 16, 16, 3, 2, "i8", "fp32", False),
    (20, 16, 65536, 1, 1, "i8", "fp32", False),       # the longest
    (20, 16, 65536, 2, 1, "bf16", "fp32", False),
    (25, 264, 40, 7, 7, "bf16", "bf16", True),        # the top-k in its own launch, just
    (24, 272, 48, 700, 8, "i8", "fp32", False),
]


@pytest.mark.parametrize("T,d,f,E,k,fmt,y_t,res", CASES)
def test_layer(T, d, f, E, k, fmt, y_t, res):
    torch = torch_mod()
    _say("moe", T, d, f, E, k, fmt, y_t, res)
    L = Layer(T, d, f, E, k, fmt)
    b = L.buffers(y_t)
    r = torch.randn(T, d, generator=L.g).to(_dt(y_t)).cuda() if res else None
    L.call(b, y_t, r)
    L.check(b, y_t, r)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
@pytest.mark.parametrize("T", [1, 6, 30])
def test_masks_slots_in_place(T, fmt):
    """Allowed experts, some rows with fewer than k; records in another order, some experts without one; y as its
    own residual."""
    torch = torch_mod()
    d, f, E, k = 512, 256, 12, 4
    _say("moe masks", T, fmt)
    L = Layer(T, d, f, E, k, fmt, 3, n_slots=9)
    m = (torch.rand(T, E, generator=L.g) < 0.6).to(torch.uint8)
    m[0] = 0
    m[0, 5] = 1  # one expert allowed
    if T > 1:
        m[1] = 0  # none
        m[2] = 1
    L.allowed = m.cuda()
    s = torch.randperm(9, generator=L.g).to(torch.int32)
    s = torch.cat([s, torch.tensor([-1, 9, -2147483648], dtype=torch.int32)])[torch.randperm(12, generator=L.g)]
    s[5] = max(int(s[5]), 0) % 9
    L.slot_of = s.cuda()
    b = L.buffers("fp32")
    r = torch.randn(T, d, generator=L.g).cuda()
    b["y"].copy_(r)
    L.call(b, "fp32", b["y"])
    L.check(b, "fp32", r)
    # no records at all: the residual
    L.n_slots = 0
    L.call(b, "fp32", r)
    torch.cuda.synchronize()
    assert torch.equal(b["y"], r)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_i8_layer_is_its_blocks(T):
    """With 8-bit records an expert's output has the bits of ft_i8_gated_ffn; the gates' sum follows in fp32."""
    torch = torch_mod()
    d, f, E, k = 1040, 784, 10, 3
    _say("moe i8 blocks", T)
    L = Layer(T, d, f, E, k, "i8", 5)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    outs = torch.empty(E, T, d, device="cuda")
    wsb = ft.ft_i8_gated_ffn_workspace_bytes(T, d, f)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    n = d * f
    for e in range(E):
        rec = L.drecs[e]
        sc = rec[3 * n:]
        m = [ft.make_i8_matrix(rec, sc, f, d), ft.make_i8_matrix(rec[n:], sc[4 * f:], f, d),
             ft.make_i8_matrix(rec[2 * n:], sc[8 * f:], d, f)]
        ft.ft_i8_gated_ffn(L.dx, d, T, ft.FT_T_BF16, ft.FT_ACT_SILU, *m, None, d, outs[e], d, ft.FT_T_FP32, ws, wsb)
    torch.cuda.synchronize()
    idx, g = b["idx"].long(), b["gates"]
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    rows = torch.arange(T, device="cuda")
    top = torch.zeros_like(want)
    for j in range(k):
        o = outs[idx[:, j], rows].double() * g[:, j:j + 1].double()
        want += o
        top += o.abs()
    # k products and additions of fp32
    assert ((b["y"].double() - want).abs() <= (k + 1) * 2.0 ** -23 * top).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
def test_captured_on_changed_inputs(fmt):
    """Captured once, replayed on other tokens between eager calls; a workspace for the most tokens serves fewer."""
    torch = torch_mod()
    _say("moe graph", fmt)
    T, d, f, E, k = 9, 512, 384, 16, 4
    L = Layer(T, d, f, E, k, fmt, 7)
    big = L.buffers("bf16", 16)
    b = L.buffers("bf16")
    b["ws"] = big["ws"]
    L.call(b, "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.call(b, "bf16")
    for i in range(4):
        L.x = torch.randn(T, d, generator=L.g).to(torch.bfloat16)
        L.dx.copy_(L.x)
        b["y"].zero_()
        b["ws"].fill_(0x3c + i)
        graph.replay()
        L.check(b, "bf16")
        other = L.buffers("bf16")
        L.call(other, "bf16")
        torch.cuda.synchronize()
        assert torch.equal(other["y"], b["y"])
        for t in (1, 4):
            few = L.buffers("bf16", t)
            few["ws"] = big["ws"]
            L.call(few, "bf16", T=t)
            # (the form goes by the number of tokens and with it the order of sums in fp32: two results of a token are each
            # within the bound of M.layer, which counts every addition's rounding in any order, not equal in bits)
            L.check(few, "bf16", T=t)
            assert torch.equal(few["idx"], b["idx"][:t])


def test_streams_at_once():
    """Layers of three formats on three streams, over and over, each with its own workspace."""
    torch = torch_mod()
    _say("moe streams")
    Ls = [Layer(T, 1024, 512, 32, 4, fmt, 9) for T, fmt in ((4, "bf16"), (11, "mxfp4"), (1, "i8"))]
    bs = [L.buffers("fp32") for L in Ls]
    for L, b in zip(Ls, bs):
        L.call(b, "fp32")
        L.check(b, "fp32")
    want = [b["y"].clone() for b in bs]
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for _ in range(20):
        for L, b, s in zip(Ls, bs, streams):
            L.call(b, "fp32", stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b["y"], w)


def test_rows_not_finite():
    """A token with a NaN keeps it to itself."""
    torch = torch_mod()
    for fmt in ("bf16", "i8"):
        _say("moe not finite", fmt)
        L = Layer(5, 256, 128, 6, 2, fmt, 11)
        L.x[3, 7] = float("nan")
        L.dx.copy_(L.x)
        b = L.buffers("fp32")
        L.call(b, "fp32")
        torch.cuda.synchronize()
        assert torch.isnan(b["y"][3]).all()
        ok = [0, 1, 2, 4]
        idx, gates = L.routed()
        assert torch.equal(b["idx"][ok], idx[ok]) and torch.equal(b["gates"][ok], gates[ok])
        want = M.layer(L.x[ok], L.recs, L.slots(), idx[ok].cpu(), gates[ok].cpu(), 256, 128, fmt, torch.float32)
        R.check(b["y"][ok], want, "y")


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
def test_rows_not_finite_among_many(fmt):
    """The same where experts have several tokens: a NaN, an infinity, and an x whose h passes the range."""
    torch = torch_mod()
    _say("moe not finite, many", fmt)
    T, d, f = 40, 512, 128
    L = Layer(T, d, f, 3, 2, fmt, 13)
    L.x[3, 7] = float("nan")
    L.x[17, 500] = float("inf")
    L.x[33] = L.x[33] * 1e30  # products near 1e31, h past 1e60
    L.dx.copy_(L.x)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    torch.cuda.synchronize()
    bad = [3, 17, 33]
    ok = [t for t in range(T) if t not in bad]
    assert not torch.isfinite(b["y"][bad]).any()
    idx, gates = L.routed()
    assert torch.equal(b["idx"][ok], idx[ok]) and torch.equal(b["gates"][ok], gates[ok])
    want = M.layer(L.x[ok], L.recs, L.slots(), idx[ok].cpu(), gates[ok].cpu(), d, f, fmt, torch.float32)
    R.check(b["y"][ok], want, "y")


def test_records_past_32_bits():
    """A record array of more than 2^32 bytes; the last experts are taken."""
    torch = torch_mod()
    _say("moe large")
    T, d, f, E, k = 3, 4096, 2048, 96, 4
    L = Layer(T, d, f, E, k, "bf16", 13, n_slots=5)
    big = torch.empty(E, L.recs.shape[1], dtype=torch.uint8, device="cuda")
    big[E - 5:] = L.drecs
    L.drecs, L.n_slots = big, E
    m = torch.zeros(T, E, dtype=torch.uint8)
    m[:, E - 5:] = 1
    L.allowed = m.cuda()
    b = L.buffers("fp32")
    L.call(b, "fp32")
    torch.cuda.synchronize()
    idx, gates = L.routed()
    assert torch.equal(b["idx"], idx) and torch.equal(b["gates"], gates) and int(idx.min()) >= E - 5
    want = M.layer(L.x, L.recs, {e: e - (E - 5) for e in range(E)}, idx.cpu(), gates.cpu(), d, f, "bf16", torch.float32)
    R.check(b["y"], want, "y")


def test_layer_with_a_shared_expert():
    """As they are used together: the routed experts added to an 8-bit shared expert's output, over two layers."""
    torch = torch_mod()
    from tests import i8_ref as I8
    _say("moe and shared")
    T, d, f, E, k = 6, 512, 384, 16, 4
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    for layer in range(2):
        L = Layer(T, d, f, E, k, "i8", 20 + layer)
        L.x = x
        L.dx.copy_(x)
        # the shared expert's weights: channels of 16 bits quantised as rows
        ws_ = []
        for N, K in ((f, d), (f, d), (d, f)):
            w = (torch.randn(N, K, generator=L.g) * K ** -0.5).to(torch.bfloat16).cuda()
            codes = torch.empty(N, K, dtype=torch.int8, device="cuda")
            scales = torch.empty(N, device="cuda")
            ft.ft_i8_quant(w, K, N, K, ft.FT_T_BF16, codes, scales)
            ws_.append((codes, scales))
        m = [ft.make_i8_matrix(c, s, *c.shape) for c, s in ws_]
        wsb = ft.ft_i8_gated_ffn_workspace_bytes(T, d, f)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        y = torch.empty(T, d, device="cuda")
        ft.ft_i8_gated_ffn(L.dx, d, T, ft.FT_T_BF16, ft.FT_ACT_SILU, *m, None, d, y, d, ft.FT_T_FP32, ws, wsb)
        shared = y.clone()
        b = L.buffers("fp32")
        b["y"] = y
        L.call(b, "fp32", y)
        L.check(b, "fp32", shared)
        R.check(shared, I8.ffn(x, *ws_, "silu", torch.bfloat16, None, torch.float32), "shared")
        x = (x.float() + y.cpu()).to(torch.bfloat16)
