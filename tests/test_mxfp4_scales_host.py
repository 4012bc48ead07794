"""Scale bytes of MXFP4 rows come in two orders, by words [words][n][16] and by
rows [n][cols/32]; of 512, 1024, ... columns both have as many bytes.  Calls
refuse the other order (and any other shape) instead of reading it."""

import pytest
import torch

from block_quantized_expert_amd import binding as B


def _tensors(n, cols):
    codes = torch.zeros(n, cols // 2, dtype=torch.uint8)
    words = torch.zeros(-(-cols // 512), n, 16, dtype=torch.uint8)
    return codes, words


@pytest.mark.parametrize("n,cols", [(4, 512), (16, 1024), (3, 4096), (2, 1024), (1, 512)])
def test_calls_refuse_scales_by_rows(n, cols):
    codes, words = _tensors(n, cols)
    rows = B.mxfp4_scale_rows(words, cols)
    assert rows.numel() == words.numel()
    weight = B.Mxfp4Weight(torch.zeros(8, cols // 2, dtype=torch.uint8),
                           torch.zeros(8, cols // 32, dtype=torch.uint8))
    shapes = [rows, words.reshape(-1), rows.view(n, -1, 16)]
    if cols > 512 and n != cols // 512:
        shapes.append(words.transpose(0, 1).contiguous())
    for bad in shapes:
        if bad.shape == words.shape:
            continue
        for call in (lambda: B.moe_dequantize_mxfp4(codes, bad),
                     lambda: B.moe_product_mxfp4(weight, codes, bad),
                     lambda: B.moe_swiglu_mxfp4(weight, weight, codes, bad)):
            with pytest.raises(ValueError, match="scales must be"):
                call()
    # in the right order the calls get as far as the device
    with pytest.raises(ValueError, match="GPU"):
        B.moe_dequantize_mxfp4(codes, words)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_product_mxfp4(weight, codes, words)


def test_scale_rows_refuse_what_is_not_words():
    _, words = _tensors(4, 1024)
    assert B.mxfp4_scale_rows(words, 1024).shape == (4, 32)
    assert B.mxfp4_scale_rows(words, 992).shape == (4, 31)
    for bad, cols in ((words, 1056), (words.reshape(4, 32), 1024),
                      (words[:1], 1024), (words[:, :, :8], 1024)):
        with pytest.raises(ValueError, match="scales must be"):
            B.mxfp4_scale_rows(bad, cols)
