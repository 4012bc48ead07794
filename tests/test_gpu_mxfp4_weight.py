"""An Mxfp4Weight serves on every stream as soon as it is made."""

import pytest
import torch

from block_quantized_expert_amd import binding as B
from test_gpu_mxfp4_tiles import _random, _words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


@pytest.mark.parametrize("on_side", [False, True])
def test_a_new_weight_serves_on_another_stream(on_side):
    # its scales are laid out behind some milliseconds of other work on the
    # stream it is made on; the product goes to a stream without any
    n, rows, cols = 40, 300, 1056
    w, x = _random(1, rows, cols, mid=124), _random(2, n, cols)
    x = x[0], _words(x[1])
    first = B.Mxfp4Weight(*w)  # kept: the new one's scales lie elsewhere
    want = B.moe_product_mxfp4(first, *x, out_dtype=torch.float32)
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    make, use = (side, None) if on_side else (torch.cuda.current_stream(), side)
    with torch.cuda.stream(make):
        for _ in range(20):
            busy @ busy
        weight = B.Mxfp4Weight(*w)
    got = B.moe_product_mxfp4(weight, *x, out_dtype=torch.float32, stream=use)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_weight_may_be_made_while_a_graph_is_captured():
    n, rows, cols = 7, 40, 544
    w, x = _random(1, rows, cols, mid=124), _random(2, n, cols)
    x = x[0], _words(x[1])
    want = B.moe_product_mxfp4(B.Mxfp4Weight(*w), *x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.moe_product_mxfp4(B.Mxfp4Weight(*w), *x)
    for i in range(3):
        got.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
