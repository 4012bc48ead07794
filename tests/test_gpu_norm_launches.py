"""The RMS norm of more rows than one launch takes: 2^21 where rows are longer
than 8192 columns (shorter ones are one launch, whose workgroups take several
rows each)."""

import pytest
import torch

from block_quantized_expert_amd import binding as B
from rows_testlib import normal

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-6
N, H = (1 << 21) + 5, 8224
AT = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, N - 2]


@pytest.fixture(scope="module")
def rows():
    """Rows alike but for a few; (x, the few, weight)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = normal(1, 1, H, dtype=BF16).cuda().repeat(N, 1)
    some = (3 * normal(2, len(AT), H)).to(BF16).cuda()
    x[AT] = some
    yield x, some, (1 + 0.2 * normal(3, H)).cuda()
    del x
    torch.cuda.empty_cache()


def _check(got, some, alike):
    """Rows AT are some's, all others alike's, which is a row."""
    assert torch.equal(got[AT], some)
    got[AT] = alike
    for part in got.split(1 << 18):
        assert bool((part == alike).all())


def test_int8(rows):
    x, some, w = rows
    q, scale = B.moe_rmsnorm_int8(x, w, EPS, scale=torch.full((N,), -1.0, device="cuda"))
    sq, ss = B.moe_rmsnorm_int8(some, w, EPS)
    aq, a = B.moe_rmsnorm_int8(x[2:3], w, EPS)
    _check(q, sq, aq)
    _check(scale, ss, a)


def test_mxfp4(rows):
    x, some, w = rows
    codes, scales = B.moe_rmsnorm_mxfp4(x, w, EPS)
    sc, ss = B.moe_rmsnorm_mxfp4(some, w, EPS)
    ac, a = B.moe_rmsnorm_mxfp4(x[2:3], w, EPS)
    _check(codes, sc, ac)
    for word in range(scales.shape[0]):
        _check(scales[word], ss[word], a[word])


def test_rows(rows):
    x, some, w = rows
    y = B.moe_rmsnorm(x, w, EPS)
    _check(y, B.moe_rmsnorm(some, w, EPS), B.moe_rmsnorm(x[2:3], w, EPS))


def test_gradients(rows):
    x, some, w = rows
    dx = B.moe_rmsnorm_backward(x, x, w, EPS, need_dweight=False)
    _check(dx, B.moe_rmsnorm_backward(some, some, w, EPS, need_dweight=False),
           B.moe_rmsnorm_backward(x[2:3], x[2:3], w, EPS, need_dweight=False))
