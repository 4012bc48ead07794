"""The RMS norm, its residual, its rounded outputs and its gradients against
64-bit references.

Bounds: the sum of squares and r are fp64.  Outputs in fp32 (and what is
rounded further) are fp64 up to one rounding: half a step.  bf16 outputs are
three fp32 roundings (r, the product with s, that with the weight) and one to
bf16.  dx = rf (w dy) - k (s rf) + dtotal in fp32: three roundings in the first
term, in the second those of k, rf, s rf and the product beside the rounding of
each w dy in k's sum, one for each of the two sums, then the output's.
dweight: two products and the rounding of r a term, one rounding for each row
that a wavefront adds, of the workgroup's part one, fp64 over the wavefronts
and the workgroups, one last rounding."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from mxfp4_testlib import norm_back_ref, norm_ref, scale_words
from mxfp4_testlib import quantize_ref as mxfp4_ref
from mxfp4_testlib import values
from rows_testlib import U32, assert_within, half_step, normal, quantize_ref, strided

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


def f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(n, h, xt, rt, wt, seed):
    x = normal(seed, n, h)
    x[:, ::97] *= 12
    res = None if rt is None else (normal(seed + 1, n, h) * 2).to(rt)
    w = (1 + 0.2 * normal(seed + 2, h)).to(wt)
    return x.to(xt), res, w


def _y_bound(ref, dtype):
    err = (3 if dtype == BF16 else 0) * U32 * np.abs(ref) * (1 + 2.0 ** -20) + 1e-14 * np.abs(ref)
    return err + half_step(dtype) * (np.abs(ref) + err) + 2.0 ** -149


# rows of one wavefront, of 4, 8 and 16 and longer, whole and ragged
SIZES = [(1, 1, 0), (1, 4096, 0), (3, 7, 1), (5, 64, 0), (6, 511, 3), (7, 512, 0), (9, 513, 0),
         (4, 1001, 1), (3, 2048, 0), (2, 2059, 0), (130, 4095, 5), (5, 4100, 0), (3, 8192, 0),
         (2, 8193, 1), (2, 16400, 0), (2, 65536, 0), (700, 96, 0)]


@pytest.mark.parametrize("xt,rt,wt,yt", [
    (BF16, None, F32, BF16), (F32, None, BF16, F32), (BF16, BF16, BF16, BF16),
    (F32, F32, F32, F32), (F32, BF16, F32, BF16), (BF16, F32, F32, F32)])
@pytest.mark.parametrize("n,h,pad", SIZES)
def test_norm(n, h, pad, xt, rt, wt, yt):
    print("case norm", n, h, pad, xt, rt, wt, yt, flush=True)
    x, res, w = _inputs(n, h, xt, rt, wt, n + h)
    y = strided(torch.zeros(n, h, dtype=yt, device="cuda"), pad).fill_(float("nan"))
    got = B.moe_rmsnorm(strided(x.cuda(), pad), w.cuda(), EPS,
                        residual=None if res is None else strided(res.cuda(), pad), y=y)
    s = x
    if res is not None:
        assert got[0] is y
        s = (x.float() + res.float()).to(rt)
        assert torch.equal(got[1].cpu(), s)
    else:
        assert got is y
    ref, _ = norm_ref(f64(s), f64(w), EPS)
    assert_within(y, ref, _y_bound(ref, yt), "y")


# so many rows that workgroups take several, one to four wavefronts a row
MANY = [(5300, 513, 0), (6001, 520, 1), (1301, 2047, 0), (1282, 2048, 3), (1290, 2049, 0),
        (1400, 2059, 1), (700, 4095, 0), (641, 4096, 0), (650, 4097, 5), (330, 8191, 1),
        (321, 8192, 0), (2051, 1031, 0), (400, 5003, 0), (260, 8189, 0)]


@pytest.mark.parametrize("xt,rt,wt,yt", [
    (BF16, None, F32, BF16), (F32, None, BF16, F32), (BF16, BF16, BF16, BF16),
    (F32, F32, F32, F32), (F32, BF16, F32, BF16), (BF16, F32, F32, F32)])
@pytest.mark.parametrize("n,h,pad", MANY)
def test_norm_of_many_rows(n, h, pad, xt, rt, wt, yt):
    test_norm(n, h, pad, xt, rt, wt, yt)


@pytest.mark.parametrize("xt,rt,wt", [(BF16, None, F32), (F32, F32, BF16), (F32, BF16, F32),
                                      (BF16, BF16, BF16)])
@pytest.mark.parametrize("n,h,pad", [(2600, 1024, 0), (5100, 544, 1), (1300, 2080, 0),
                                     (700, 4064, 3), (650, 4128, 0), (330, 8160, 0)])
def test_rounded_outputs_of_many_rows(n, h, pad, xt, rt, wt):
    test_rounded_outputs_are_the_quantizers_on_the_fp32_output(n, h, pad, xt, rt, wt)


@pytest.mark.parametrize("n,h", [(3, 5), (4, 513), (9, 1001), (5, 8201), (700, 4097), (5300, 519),
                                 (1400, 2053)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_total_may_be_the_residual_at_odd_sizes(n, h, dtype):
    x, res, w = (t.cuda() for t in _inputs(n, h, dtype, dtype, F32, h))
    want = B.moe_rmsnorm(x, w, EPS, residual=res)
    assert torch.equal(want[1], (x.float() + res.float()).to(dtype))
    r = strided(res, 3).clone() if n < 10 else res.clone()
    y, total = B.moe_rmsnorm(x, w, EPS, residual=r, total=r)
    assert total is r and torch.equal(r, want[1]) and torch.equal(y, want[0])


@pytest.mark.parametrize("xt,rt,wt", [(BF16, None, F32), (F32, F32, BF16), (F32, BF16, F32),
                                      (BF16, BF16, BF16)])
@pytest.mark.parametrize("n,h,pad", [(1, 32, 0), (1, 4096, 0), (6, 480, 1), (7, 512, 0), (9, 544, 0),
                                     (4, 992, 1), (3, 2048, 0), (2, 2080, 0), (130, 4064, 5),
                                     (3, 8192, 0), (2, 8224, 1), (2, 16416, 0), (1, 65536, 0),
                                     (500, 96, 0)])
def test_rounded_outputs_are_the_quantizers_on_the_fp32_output(n, h, pad, xt, rt, wt):
    print("case rounded", n, h, pad, xt, rt, wt, flush=True)
    x, res, w = _inputs(n, h, xt, rt, wt, n + h)
    xd, wd = strided(x.cuda(), pad), w.cuda()
    rd = None if res is None else strided(res.cuda(), pad)
    kw = dict(residual=rd)
    y, *total = (lambda r: r if isinstance(r, tuple) else (r,))(
        B.moe_rmsnorm(xd, wd, EPS, y_dtype=F32, **kw))
    q, scale, *t8 = B.moe_rmsnorm_int8(xd, wd, EPS, **kw)
    codes, words, *t4 = B.moe_rmsnorm_mxfp4(xd, wd, EPS, **kw)
    for t in (t8, t4):
        assert len(t) == len(total) and all(torch.equal(a, b) for a, b in zip(t, total))
    for got, want in zip((q, scale), B.moe_quantize_int8(y)):
        assert torch.equal(got, want)
    for got, want in zip((codes, words), B.moe_quantize_mxfp4(y)):
        assert torch.equal(got, want)
    # and those are the definitions', of values that are the reference's up to a rounding
    yn = f64(y)
    ref, _ = norm_ref(f64(x if res is None else total[0]), f64(w), EPS)
    assert_within(y, ref, _y_bound(ref, F32), "y")
    rq, rs = quantize_ref(yn)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(scale.cpu().numpy(), rs)
    rc, rb = mxfp4_ref(yn)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(words.cpu().numpy(), scale_words(rb))


def test_one_row_at_a_time_gives_the_same_bits():
    x, res, w = (t.cuda() for t in _inputs(37, 4096, BF16, BF16, F32, 3))
    y, total = B.moe_rmsnorm(x, w, EPS, residual=res)
    q, scale, _ = B.moe_rmsnorm_int8(x, w, EPS, residual=res)
    for i in (0, 1, 17, 36):
        yi, ti = B.moe_rmsnorm(x[i:i + 1], w, EPS, residual=res[i:i + 1])
        qi, si, _ = B.moe_rmsnorm_int8(x[i:i + 1], w, EPS, residual=res[i:i + 1])
        assert torch.equal(yi[0], y[i]) and torch.equal(ti[0], total[i])
        assert torch.equal(qi[0], q[i]) and torch.equal(si[0], scale[i])


@pytest.mark.parametrize("h", [96, 2048, 4096, 9000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_total_may_be_the_residual(h, dtype):
    x, res, w = (t.cuda() for t in _inputs(5, h, dtype, dtype, F32, h))
    want = B.moe_rmsnorm(x, w, EPS, residual=res)
    r = res.clone()
    y, total = B.moe_rmsnorm(x, w, EPS, residual=r, total=r)
    assert total is r and torch.equal(r, want[1]) and torch.equal(y, want[0])
    if h % 32 == 0:
        want = B.moe_rmsnorm_mxfp4(x, w, EPS, residual=res)
        r = res.clone()
        got = B.moe_rmsnorm_mxfp4(x, w, EPS, residual=r, total=r)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_zero_large_and_non_finite_rows():
    h = 512
    x = normal(1, 8, h)
    x[1] = 0
    x[2] *= 1e25       # squares leave fp32
    x[3] *= 1e-30      # far below eps
    x[4, 5] = float("inf")
    x[5, 511] = float("nan")
    x[6, 0], x[6, 1] = float("-inf"), float("nan")
    w = (1 + 0.2 * normal(2, h))
    keep = [0, 1, 2, 3, 7]
    ref, _ = norm_ref(f64(x[keep]), f64(w), EPS)
    y = B.moe_rmsnorm(x.cuda(), w.cuda(), EPS)
    assert_within(y[keep], ref, _y_bound(ref, F32), "y")
    y = y.cpu()
    assert torch.isnan(y[4, 5]) and not y[4, :5].any() and not y[4, 6:].any()  # s * 0
    assert torch.isnan(y[5]).all() and torch.isnan(y[6]).all()
    q, scale = (t.cpu() for t in B.moe_rmsnorm_int8(x.cuda(), w.cuda(), EPS))
    assert torch.isnan(scale[4:7]).all() and not q[4:7].any() and not q[1].any() and scale[1] == 0
    codes, words = B.moe_rmsnorm_mxfp4(x.cuda(), w.cuda(), EPS)
    back = B.moe_dequantize_mxfp4(codes, words, F32).cpu()
    assert torch.isnan(back[4, :32]).all() and not back[4, 32:].any()
    assert torch.isnan(back[5:7]).all() and not back[1].any()
    assert torch.isfinite(back[keep]).all()


@pytest.mark.parametrize("out", ["rows", "int8", "mxfp4"])
def test_more_rows_than_a_launch_takes(out):
    # rows go in launches of 2^21
    n, h = (1 << 21) + 5, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, h, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(h, generator=g, device="cuda")
    at = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, n - 1]
    if out == "rows":
        y = B.moe_rmsnorm(x, w, EPS, y=torch.full((n, h), float("nan"), device="cuda"))
        assert not torch.isnan(y).any()
        ref, _ = norm_ref(f64(x[at]), f64(w), EPS)
        assert_within(y[at], ref, _y_bound(ref, F32), "y")
    elif out == "int8":
        q, s = B.moe_rmsnorm_int8(x, w, EPS, scale=torch.full((n,), -1.0, device="cuda"))
        assert bool((s > 0).all())
        qa, sa = B.moe_rmsnorm_int8(x[at], w, EPS)
        assert torch.equal(q[at], qa) and torch.equal(s[at], sa)
    else:
        c, s = B.moe_rmsnorm_mxfp4(x, w, EPS,
                                   scales=torch.full((1, n, 16), 99, dtype=torch.uint8,
                                                     device="cuda"))
        assert not s[0, :, 1:].any() and bool((s[0, :, 0] > 100).all())
        ca, sa = B.moe_rmsnorm_mxfp4(x[at], w, EPS)
        assert torch.equal(c[at], ca) and torch.equal(s[:, at], sa)


# ------------------------------------------------------------- gradients


def _back_check(n, h, pad, dt, st, wt, total):
    s, _, w = _inputs(n, h, st, None, wt, n + h)
    dy = normal(n + h + 5, n, h).to(dt)
    tot = normal(n + h + 6, n, h).to(st) if total else None
    got = B.moe_rmsnorm_backward(strided(dy.cuda(), pad), strided(s.cuda(), pad), w.cuda(), EPS,
                                 dtotal=None if tot is None else strided(tot.cuda(), pad),
                                 dx=strided(torch.zeros(n, h, dtype=st, device="cuda"), pad))
    sn, wn, dn = f64(s), f64(w), f64(dy)
    tn = None if tot is None else f64(tot)
    dx, dw = norm_back_ref(dn, sn, wn, EPS, tn)
    _, r = norm_ref(sn, wn, EPS)
    g = wn * dn
    k = np.abs(r ** 3 * (sn * g).mean(axis=1, keepdims=True))
    kerr = U32 * (np.abs(sn * g).mean(axis=1, keepdims=True) * r ** 3 + k)
    err = 3 * U32 * np.abs(r * g) + np.abs(sn) * (kerr + 3 * U32 * k)
    sums = np.abs(r * g) + np.abs(k * sn) + (0 if tn is None else np.abs(tn) + np.abs(dx))
    err = (err + U32 * sums) * (1 + 2.0 ** -10)
    assert_within(got[0], dx, err + half_step(st) * (np.abs(dx) + err) + 2.0 ** -149, "dx")
    terms = np.abs(dn * sn * r).sum(axis=0)
    groups = max(1, B.lib().moe_rmsnorm_backward_workspace_bytes(n, h) // (4 * h))
    rows = -(-n // groups) + 1
    assert_within(got[1], dw, U32 * ((3 + rows + 3) * terms + np.abs(dw)) * (1 + 2.0 ** -10),
                  "dweight")
    return got


@pytest.mark.parametrize("dt,st,wt,total", [
    (BF16, BF16, F32, True), (F32, F32, F32, False), (BF16, F32, BF16, True),
    (F32, BF16, F32, False), (F32, F32, BF16, True)])
@pytest.mark.parametrize("n,h,pad", SIZES + [(1300, 256, 0), (1025, 4096, 0), (600, 8192, 0),
                                             (2500, 40, 1), (70, 8200, 0)])
def test_gradients(n, h, pad, dt, st, wt, total):
    print("case gradients", n, h, pad, dt, st, wt, total, flush=True)
    _back_check(n, h, pad, dt, st, wt, total)


# rows by the thousand: one to sixteen wavefronts a row, several rows at once
@pytest.mark.parametrize("dt,st,wt,total", [
    (BF16, BF16, F32, True), (F32, F32, F32, False), (BF16, F32, BF16, True),
    (BF16, BF16, BF16, False), (F32, F32, BF16, True)])
@pytest.mark.parametrize("n,h,pad", [(1537, 513, 0), (1600, 1031, 1), (1701, 2053, 0),
                                     (1541, 4099, 0), (1600, 8191, 0), (4200, 1024, 0),
                                     (5003, 9, 1), (520, 517, 0), (1536, 1025, 0),
                                     (1801, 5119, 0), (1702, 5123, 1), (1600, 6200, 0)])
def test_gradients_of_many_rows(n, h, pad, dt, st, wt, total):
    print("case gradients", n, h, pad, dt, st, wt, total, flush=True)
    _back_check(n, h, pad, dt, st, wt, total)


@pytest.mark.parametrize("n,h", [(3, 5), (9, 1001), (5, 8201), (1600, 1025), (1601, 4097)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_into_dtotal_at_odd_sizes(n, h, dtype):
    s, _, w = (t if t is None else t.cuda() for t in _inputs(n, h, dtype, None, F32, h))
    dy, tot = normal(1, n, h, dtype=dtype).cuda(), normal(2, n, h, dtype=dtype).cuda()
    dx, dw = B.moe_rmsnorm_backward(dy, s, w, EPS, dtotal=tot)
    got = B.moe_rmsnorm_backward(dy, s, w, EPS, dtotal=tot, dx=tot)
    assert got[0] is tot and torch.equal(tot, dx) and torch.equal(got[1], dw)


def test_short_rows_of_more_than_a_launch():
    # rows of fewer than eight columns go in launches of 2^21, with their gradients
    n, h = (1 << 21) + 5, 3
    x = torch.arange(n * h, device="cuda").remainder(13).sub(6).float().view(n, h)
    x[:, 0] += 0.5
    w = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    y = B.moe_rmsnorm(x, w, EPS)
    at = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, n - 1]
    ref, _ = norm_ref(f64(x[at]), f64(w), EPS)
    assert_within(y[at], ref, _y_bound(ref, F32), "y")
    total = torch.empty_like(x)
    y2, t2 = B.moe_rmsnorm(x, w, EPS, residual=torch.zeros_like(x), total=total)
    assert t2 is total and torch.equal(total, x) and torch.equal(y2, y)
    dx, dw = B.moe_rmsnorm_backward(x, x, w, EPS)
    want, _ = norm_back_ref(f64(x[at]), f64(x[at]), f64(w), EPS)
    # each of dx's terms is below 2^5 and rounded four times
    assert_within(dx[at], want, 4 * U32 * 2.0 ** 5, "dx")
    _, dwr = norm_back_ref(f64(x), f64(x), f64(w), EPS)
    rows = -(-n // 64) + 1
    assert_within(dw, dwr, U32 * (6 + rows) * (f64(x) ** 2 * norm_ref(f64(x), 1.0, EPS)[1]).sum(0),
                  "dweight")


@pytest.mark.parametrize("n,h", [(6, 1000), (700, 1000), (1600, 520), (6, 9000)])
@pytest.mark.parametrize("scale", [2.0 ** 84, 2.0 ** 110, 2.0 ** -100])
def test_gradients_of_far_rows(n, h, scale):
    # r from 2^-110 to 2^10: squares, r^3 and dy s of large rows leave fp32.  dx
    # of those is of the order of r; times 1 / r it is held to the bound of rows
    # of order one (4 roundings of each of two terms and the sum, and the w dy
    # in k's sum: 20 U32 of values below 64)
    s, _, w = _inputs(n, h, F32, None, F32, h)
    s = s * scale
    dy = normal(3, n, h) * 64
    dx, dw = B.moe_rmsnorm_backward(dy.cuda(), s.cuda(), w.cuda(), EPS)
    want, dwr = norm_back_ref(f64(dy), f64(s), f64(w), EPS)
    _, r = norm_ref(f64(s), f64(w), EPS)
    size = np.abs(f64(w) * f64(dy)) + np.abs(f64(s) * r) * np.abs(
        (f64(s) * r * f64(w) * f64(dy))).mean(axis=1, keepdims=True)
    assert np.all(np.abs(f64(dx) - want) / r <= 20 * U32 * size + 2.0 ** -149 / r)
    terms = np.abs(f64(dy) * f64(s) * r).sum(axis=0)
    assert_within(dw, dwr, U32 * ((n + 9) * terms + np.abs(dwr)) + 2.0 ** -149, "dweight")


def test_gradients_against_differences():
    # L = sum(dy * n(x)) in 64 bits; a central difference of step d is off by
    # d^2 / 6 times the third derivative (of order 1 here) and 2^-53 L / d: with
    # d = 2^-14 both are below 1e-8.  The kernel's own error is a few U32 of
    # values of order 1.
    n, h = 3, 24
    x, w, dy = normal(1, n, h), 1 + 0.2 * normal(2, h), normal(3, n, h)
    dx, dw = B.moe_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), EPS)
    xn, wn, dn = f64(x), f64(w), f64(dy)

    def loss(x, w):
        return (dn * norm_ref(x, w, EPS)[0]).sum()

    d = 2.0 ** -14
    for i in range(n):
        for j in range(h):
            step = np.zeros((n, h))
            step[i, j] = d
            diff = (loss(xn + step, wn) - loss(xn - step, wn)) / (2 * d)
            assert abs(diff - float(dx[i, j])) <= 2e-6
    for j in range(h):
        step = np.zeros(h)
        step[j] = d
        diff = (loss(xn, wn + step) - loss(xn, wn - step)) / (2 * d)
        assert abs(diff - float(dw[j])) <= 2e-6


@pytest.mark.parametrize("h", [96, 1024, 4096, 8192, 9000])
def test_gradients_without_weights_and_into_dtotal(h):
    n = 9
    s, _, w = (t if t is None else t.cuda() for t in _inputs(n, h, F32, None, F32, h))
    dy, tot = normal(1, n, h).cuda(), normal(2, n, h).cuda()
    dx, dw = B.moe_rmsnorm_backward(dy, s, w, EPS, dtotal=tot)
    alone = B.moe_rmsnorm_backward(dy, s, w, EPS, dtotal=tot, need_dweight=False)
    assert torch.equal(alone, dx)
    t = tot.clone()
    got = B.moe_rmsnorm_backward(dy, s, w, EPS, dtotal=t, dx=t)
    assert got[0] is t and torch.equal(t, dx) and torch.equal(got[1], dw)


def test_no_rows():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    assert B.moe_rmsnorm(x, w).shape == (0, 64)
    assert [tuple(t.shape) for t in B.moe_rmsnorm(x, w, residual=x)] == [(0, 64)] * 2
    assert [tuple(t.shape) for t in B.moe_rmsnorm_int8(x, w)] == [(0, 64), (0,)]
    assert [tuple(t.shape) for t in B.moe_rmsnorm_mxfp4(x, w)] == [(0, 32), (1, 0, 16)]
    dx, dw = B.moe_rmsnorm_backward(x, x, w, dweight=torch.full((64,), 7.0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


def test_rows_past_32_bit_offsets():
    # 40000 rows of 65536: the last lie past 2^31 elements; some rows are looked at
    n, h = 40000, 65536
    x = torch.ones((n, h), dtype=BF16, device="cuda")
    at = torch.tensor([0, 32767, 32768, 39999])
    some = normal(5, 4, h, dtype=BF16)
    x[at.cuda()] = some.cuda()
    w = (1 + 0.2 * normal(6, h))
    y = B.moe_rmsnorm(x, w.cuda(), EPS)
    ref, _ = norm_ref(f64(some), f64(w), EPS)
    assert_within(y[at.cuda()], ref, _y_bound(ref, BF16), "y")
    dx, dw = B.moe_rmsnorm_backward(x, x, w.cuda(), EPS)
    look = f64(some)
    want, _ = norm_back_ref(look, look, f64(w), EPS)
    assert_within(dx[at.cuda()], want, 2 * half_step(BF16) * np.abs(want) + 1e-4, "dx")
    # a row of ones and dy = 1: dweight_j = n r, the looked at rows beside
    _, r = norm_ref(look, f64(w), EPS)
    dwr = (n - 4) / np.sqrt(1 + EPS) + (look * look * r).sum(axis=0)
    assert_within(dw, dwr, U32 * 700 * dwr, "dweight")
    del x, y, dx
    torch.cuda.empty_cache()


def test_results_repeat_on_another_stream_and_in_a_graph():
    n, h = 600, 1024
    x, res, w = (t.cuda() for t in _inputs(n, h, BF16, BF16, F32, 1))
    dy = normal(9, n, h, dtype=BF16).cuda()

    def passes(stream=None):
        y, total = B.moe_rmsnorm(x, w, EPS, residual=res, stream=stream)
        q, s, _ = B.moe_rmsnorm_int8(x, w, EPS, residual=res, stream=stream)
        c, z, _ = B.moe_rmsnorm_mxfp4(x, w, EPS, residual=res, stream=stream)
        dx, dw = B.moe_rmsnorm_backward(dy, total, w, EPS, dtotal=dy, stream=stream)
        return y, total, q, s, c, z, dx, dw

    want = [t.clone() for t in passes()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = passes(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = passes()
    for i in range(4):
        x.mul_(1.25)
        want = [t.clone() for t in passes()]
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_gradients_on_two_streams_at_once():
    # each call has a workspace of its own
    n, h = 3001, 1031
    s, _, w = (t if t is None else t.cuda() for t in _inputs(n, h, BF16, None, F32, 1))
    dys = [normal(9 + i, n, h, dtype=BF16).cuda() for i in range(2)]
    want = [B.moe_rmsnorm_backward(dy, s, w, EPS) for dy in dys]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[B.moe_rmsnorm_backward(dy, s, w, EPS, stream=st) for dy, st in zip(dys, streams)]
           for _ in range(4)]
    torch.cuda.synchronize()
    for both in got:
        for a, b in zip(both, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals_on_the_gpu():
    x, w = torch.zeros(4, 48, device="cuda"), torch.ones(48, device="cuda")
    with pytest.raises(B.MoeError) as e:
        B.moe_rmsnorm_mxfp4(x, w)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED and "moe_rmsnorm_mxfp4" in str(e.value)
    with pytest.raises(B.MoeError):
        B.moe_rmsnorm_int8(x[:, :40].contiguous(), w[:40])
    with pytest.raises(B.MoeError) as e:
        B.moe_rmsnorm(x, w, 0.0)
    assert e.value.status == B.MOE_ERR_INVALID
    with pytest.raises(ValueError, match="weight must be"):
        B.moe_rmsnorm(x, w[:40])
    with pytest.raises(ValueError, match="total needs a residual"):
        B.moe_rmsnorm(x, w, total=x.clone())
    with pytest.raises(ValueError, match="total must have the residual's dtype"):
        B.moe_rmsnorm(x, w, residual=x, total=x.bfloat16())
    with pytest.raises(ValueError, match="dtotal must have s's dtype"):
        B.moe_rmsnorm_backward(x, x, w, dtotal=x.bfloat16())
    with pytest.raises(ValueError, match="expected cuda"):
        B.moe_rmsnorm(x, w, residual=x.cpu())
    torch.cuda.synchronize()


def test_values_helper_is_the_dequantizer():
    x = normal(4, 5, 96)
    codes, words = B.moe_quantize_mxfp4(x.cuda())
    b = B.mxfp4_scale_rows(words, 96).cpu().numpy()
    assert np.array_equal(f64(B.moe_dequantize_mxfp4(codes, words, F32)),
                          values(codes.cpu().numpy(), b))
