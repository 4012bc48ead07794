"""dweight of the RMS norm for rows that are not kept in registers (more than
8192 columns, or fewer than eight): summed over the rows in fp64.

Bound: a term is dy times s r with r and s r rounded to fp32, two half-steps;
sums are fp64 but for one rounding of each of the 64 parts and the last one.
So four half-steps of the terms' magnitudes, whatever the number of rows."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from mxfp4_testlib import norm_ref
from rows_testlib import U32, assert_within, normal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt,st", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,h", [(1, 8193), (63, 3), (64, 1), (65, 8200), (40000, 7), ((1 << 20) + 3, 5),
                                 (3001, 8200), (700, 16385)])
def test_dweight_of_rows_alike(n, h, dt, st):
    # a term that is the same in every row: each addition to an fp32 sum would be
    # rounded the same way, so that n / 64 of them add up to far more than the bound
    print("case dweight", n, h, dt, st, flush=True)
    s, dy = (normal(3, 1, h).abs() + 0.3).to(st), (normal(4, 1, h).abs() + 0.3).to(dt)
    w = 1 + 0.2 * normal(5, h)
    _, dw = B.moe_rmsnorm_backward(dy.cuda().repeat(n, 1), s.cuda().repeat(n, 1), w.cuda(), EPS)
    _, r = norm_ref(s.double().numpy(), w.double().numpy(), EPS)
    want = n * (dy.double().numpy() * s.double().numpy() * r)[0]
    assert_within(dw, want, 4 * U32 * want * (1 + 2.0 ** -20), "dweight")


@pytest.mark.parametrize("n,h", [(70001, 4), (2100, 9001)])
def test_dweight_of_rows_of_both_signs(n, h):
    print("case signs", n, h, flush=True)
    s, dy, w = normal(1, n, h), normal(2, n, h) + 0.25, 1 + 0.2 * normal(5, h)
    _, dw = B.moe_rmsnorm_backward(dy.cuda(), s.cuda(), w.cuda(), EPS)
    sn, dn = s.double().numpy(), dy.double().numpy()
    _, r = norm_ref(sn, w.double().numpy(), EPS)
    terms = dn * sn * r
    assert_within(dw, terms.sum(axis=0), 4 * U32 * np.abs(terms).sum(axis=0) * (1 + 2.0 ** -20),
                  "dweight")
