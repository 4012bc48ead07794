"""Tiled MXFP4 products with reductions long enough that the copies' buffers and
the slots of the scale words are used again within a tile, dense and grouped,
gathered and in expert order, plain and with SwiGLU, in both output types.
References and bounds as in test_gpu_mxfp4_tiles.py."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from test_gpu_mxfp4_tiles import (_out, _product, _random, _within, _within_swiglu, _words,
                                  counts_of)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# rows of the left operand, weight rows, cols: 9, 16 and 17 steps of 256 inputs, 5, 8
# and 9 words of scales, the last step whole or a part
DENSE = [
    (35, 8137, 2080), (35, 6889, 4096), (33, 7465, 4128), (257, 6855, 2080), (1065, 7187, 2080),
    (6622, 2447, 2080), (260, 6625, 4096), (258, 6971, 4128), (5980, 1297, 4096),
    (2309, 3357, 4128), (6671, 2317, 2080), (2314, 6793, 4096), (2324, 6823, 4128),
    (519, 6611, 4096), (647, 5641, 4128), (130, 5671, 2080), (130, 5457, 4128), (135, 5723, 4096),
    (259, 5937, 2080), (4386, 3589, 4096), (3378, 4721, 4128), (3925, 8099, 2080),
    (7968, 3861, 4096), (3873, 8121, 4128),
]
# experts, slots, weight rows, cols
GROUPED = [
    (24, 42, 6401, 2080), (24, 42, 7065, 4096), (24, 60, 6707, 4128), (12, 449, 6117, 2080),
    (12, 339, 5495, 4128), (24, 643, 2789, 4096), (40, 1158, 1303, 2080), (64, 6424, 787, 2080),
    (40, 1074, 1429, 4128), (40, 1241, 1333, 4096), (64, 6093, 887, 4096), (24, 4560, 2917, 2080),
    (64, 7131, 801, 4128), (12, 3422, 3871, 4096), (64, 6625, 411, 2080), (12, 3582, 3933, 4128),
    (64, 5891, 425, 4128), (64, 6234, 437, 4096), (12, 3000, 7957, 2080), (24, 741, 6247, 2080),
    (24, 505, 6101, 4096), (24, 543, 6073, 4128), (12, 3862, 6603, 4096), (12, 4509, 5851, 4128),
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


def _weights(e, rows, cols):
    w, u = (_random(i, e, rows, cols, mid=124) for i in (1, 2))
    return w, u, B.Mxfp4Weight(*w), B.Mxfp4Weight(*u)


def _check(gw, gu, left, a, b, grouping=None, top_k=0):
    """Both products in both types against a (gate's reference and error) and b
    (up's); the rows behind the last expert's are 0, the gaps between rows kept."""
    n, rows = a[0].shape
    total = n if grouping is None else int(grouping[1][-1])
    for dtype in (BF16, F32):
        out, gap = _out(n, rows, dtype, dtype == BF16)
        B.moe_product_mxfp4(gw, *left, grouping, top_k=top_k, out=out)
        _within(out, *a, "product")
        assert bool((gap == 7).all()) and not bool(out[total:].any())
        out, gap = _out(n, rows, dtype, dtype == F32)
        B.moe_swiglu_mxfp4(gw, gu, *left, grouping, top_k=top_k, out=out)
        _within_swiglu(out, *a, *b, "swiglu")
        assert bool((gap == 7).all()) and not bool(out[total:].any())


@pytest.mark.parametrize("n,rows,cols", DENSE)
def test_dense_products_of_long_reductions(n, rows, cols):
    print("case dense", n, rows, cols, flush=True)
    w, u, gw, gu = _weights(1, rows, cols)
    x = _random(3, n, cols)
    every = torch.arange(n, device="cuda")
    _check(gw, gu, (x[0], _words(x[1])), _product(w, x, [0, n], every),
           _product(u, x, [0, n], every))


@pytest.mark.parametrize("e,slots,rows,cols", GROUPED)
def test_grouped_products_of_long_reductions(e, slots, rows, cols):
    print("case grouped", e, slots, rows, cols, flush=True)
    k = 3 if slots % 3 == 0 else 2 if slots % 2 == 0 else 1
    counts = counts_of(e, slots)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = int(offsets[-1])
    perm = np.random.default_rng(slots).permutation(slots).astype(np.int32)
    g = tuple(torch.from_numpy(v).cuda() for v in (counts.astype(np.int32), offsets, perm, perm))
    w, u, gw, gu = _weights(e, rows, cols)
    x = _random(3, slots // k, cols)
    left = torch.div(g[2].long(), k, rounding_mode="floor")
    _check(gw, gu, (x[0], _words(x[1])), _product(w, x, offsets, left),
           _product(u, x, offsets, left), g, k)
    x = _random(4, slots, cols)
    every = torch.arange(slots, device="cuda")
    a, b = _product(w, x, offsets, every), _product(u, x, offsets, every)
    x[1][total:] = 255  # rows that nothing may read
    _check(gw, gu, (x[0], _words(x[1])), a, b, g)
