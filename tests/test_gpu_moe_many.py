"""GPU tests of the routed layer where experts have several tokens (the matrix form, its top-k in a launch of its own past 24
tokens, its joins where blocks share rows of y): captured and replayed, and beside other streams."""
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_moe_layer import Layer, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
@pytest.mark.parametrize("T,d,f,E,k", [(40, 512, 384, 6, 3), (64, 2304, 256, 8, 4), (18, 1024, 256, 3, 2)])
def test_captured_on_changed_inputs(T, d, f, E, k, fmt):
    """Replayed on other tokens between eager calls on another workspace, its own filled anew: equal bits."""
    torch = torch_mod()
    _say("moe many, graph", T, d, f, E, k, fmt)
    L = Layer(T, d, f, E, k, fmt, 41)
    b = L.buffers("fp32")
    r = torch.randn(T, d, generator=L.g).cuda()
    L.call(b, "fp32", r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.call(b, "fp32", r)
    for i in range(4):
        L.x = torch.randn(T, d, generator=L.g).to(torch.bfloat16)
        L.dx.copy_(L.x)
        b["y"].zero_()
        b["idx"].fill_(-9)
        b["ws"].fill_(0x3c + i)
        graph.replay()
        L.check(b, "fp32", r)
        other = L.buffers("fp32")
        L.call(other, "fp32", r)
        torch.cuda.synchronize()
        for n in ("y", "idx", "gates"):
            assert torch.equal(other[n], b[n]), n


def test_streams_at_once():
    """Each format on two streams, rows of y shared and not, over and over, each with its own workspace."""
    torch = torch_mod()
    _say("moe many, streams")
    Ls = [Layer(T, d, 384, E, k, fmt, 43) for fmt in ("bf16", "mxfp4", "i8")
          for T, d, E, k in ((40, 512, 6, 3), (64, 2304, 8, 4))]
    bs = [L.buffers("fp32") for L in Ls]
    for L, b in zip(Ls, bs):
        L.call(b, "fp32")
        L.check(b, "fp32")
    want = [b["y"].clone() for b in bs]
    for b in bs:
        b["y"].zero_()
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for _ in range(12):
        for L, b, s in zip(Ls, bs, streams):
            L.call(b, "fp32", stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b["y"], w)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4", "i8"])
def test_two_graphs_on_their_own_workspaces(fmt):
    """Two captured layers replayed in turn and at once."""
    torch = torch_mod()
    _say("moe many, two graphs", fmt)
    Ls = [Layer(T, 512, 256, 5, 3, fmt, s) for T, s in ((36, 45), (30, 46))]
    bs = [L.buffers("bf16") for L in Ls]
    graphs = []
    for L, b in zip(Ls, bs):
        L.call(b, "bf16")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.call(b, "bf16")
        graphs.append(g)
    want = [b["y"].clone() for b in bs]
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for i in range(6):
        for b in bs:
            b["y"].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if i % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for L, b, w in zip(Ls, bs, want):
            assert torch.equal(b["y"], w)
    for L, b in zip(Ls, bs):
        L.check(b, "bf16")
