"""Scale words given as outputs are looked at by shape, as those given as inputs."""

import pytest
import torch

from block_quantized_expert_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def test_outputs_by_rows_are_refused():
    # returned before anything is enqueued
    n, c = 6, 1024
    x, w = torch.randn(n, c, device="cuda"), torch.ones(c, device="cuda")
    words = torch.full((2, n, 16), 77, dtype=torch.uint8, device="cuda")
    for bad in (words.view(n, 32), words.view(-1), words.view(n, 2, 16)):
        with pytest.raises(ValueError, match="scales must be"):
            B.moe_quantize_mxfp4(x, scales=bad)
        with pytest.raises(ValueError, match="scales must be"):
            B.moe_rmsnorm_mxfp4(x, w, scales=bad)
    torch.cuda.synchronize()
    assert bool((words == 77).all())
    codes, got = B.moe_quantize_mxfp4(x, scales=words)
    assert got is words
    want = B.moe_dequantize_mxfp4(codes, words)
    rows = B.mxfp4_scale_rows(words, c)
    with pytest.raises(ValueError, match="scales must be"):
        B.moe_dequantize_mxfp4(codes, rows)
    # the words that rows make, by way of a weight, are the same
    weight = B.Mxfp4Weight(codes, rows)
    assert torch.equal(B.moe_dequantize_mxfp4(codes, weight.scales[0]), want)
