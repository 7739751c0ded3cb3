"""GPU test: the routed layer writes x in the order of its rows' form only where that form reads it."""
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_moe_layer import Layer, _say

pytestmark = pytest.mark.gpu


def test_matrix_form_leaves_the_planes():
    """64 tokens of 4 experts in MXFP4: the workspace keeps at least as many bytes as the planes of x take."""
    torch = torch_mod()
    _say("moe planes")
    L = Layer(64, 2304, 128, 4, 4, "mxfp4", 61)
    b = L.buffers("fp32")
    L.call(b, "fp32")
    L.check(b, "fp32")
    assert int((b["ws"] == 0xa5).sum()) >= L.T * L.d * 2
