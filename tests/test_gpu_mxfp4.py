"""Rounding to MXFP4 and back, and the MXFP4 products against 64-bit
references.

Bounds: codes, scale bytes and the values they stand for are exact.  A
product's terms are exact in fp32 (two E2M1 values have four bits together).
With `unit` the smallest nonzero term that the row's and the channel's scales
allow, every partial sum is a multiple of it, so where the sum of the terms'
magnitudes is below 2^24 units every sum in fp32 is exact, in any order; where
it is not, each of the at most cols / 32 + 8 additions is off by at most 2^-20
of the magnitudes' sum.  Half a step of the output's type comes on top.
SwiGLU's quotient g / (1 + e^-g) has condition number 1 + |g| in g and |g| / (1 +
e^g) <= 1 / 4 + |g| in the exponential's argument (the hardware's adds 2 |g| half
steps); the exponential, the sum, the quotient and the last product are some
ten half-steps."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from mxfp4_testlib import quantize_ref, random_mxfp4, scale_words, values
from rows_testlib import U32, assert_within, group, half_step, make_ids, normal, on_gpu, strided

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


# ------------------------------------------------------- rounding and back


def _check_quantize(x, pad=0):
    n, c = x.shape
    xd = strided(x.cuda(), pad)
    words = -(-c // 512)
    codes = torch.full((n, c // 2), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((words, n, 16), 77, dtype=torch.uint8, device="cuda")
    got = B.moe_quantize_mxfp4(xd, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    rc, rb = quantize_ref(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), scale_words(rb))
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(B.mxfp4_scale_rows(scales, c).cpu().numpy(), rb)
    v = values(rc, rb)
    for dtype in (F32, BF16):
        back = strided(torch.zeros(n, c, dtype=dtype, device="cuda"), pad).fill_(7.0)
        assert B.moe_dequantize_mxfp4(codes, scales, x=back) is back
        assert np.array_equal(back.double().cpu().numpy(), v, equal_nan=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,c,pad", [
    (1, 32, 0), (1, 4096, 0), (17, 32, 1), (33, 64, 0), (7, 96, 3), (9, 128, 0), (5, 160, 0),
    (21, 256, 1), (3, 480, 0), (4, 512, 0), (6, 544, 5), (130, 1024, 0), (3, 2080, 7),
    (2, 65536, 0), (700, 4096, 0)])
def test_rounding_is_exact_both_ways(n, c, pad, dtype):
    print("case quantize", n, c, pad, dtype, flush=True)
    x = normal(n + c, n, c)
    x[:, ::97] *= 12
    # blocks of every magnitude
    x *= torch.exp2(torch.arange(n * c // 32).reshape(n, -1).float() % 61 - 30).repeat_interleave(
        32, dim=1)
    _check_quantize(x.to(dtype), pad)


# so many bf16 columns that a wavefront takes several words
@pytest.mark.parametrize("n,c,pad", [(8201, 1056, 0), (37700, 224, 1), (2051, 4128, 0),
                                     (263001, 32, 0), (129, 65536, 3)])
def test_rounding_of_many_rows(n, c, pad):
    print("case quantize many", n, c, pad, flush=True)
    x = normal(n + c, n, c)
    x[:, ::97] *= 12
    x[n // 2, 5] = float("inf")
    _check_quantize(x.bfloat16(), pad)


def test_borders_and_far_values():
    # the borders of E2M1 under every scale, their neighbours in fp32, and what saturates
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = []
    for e in list(range(-125, 126, 10)) + [-125, -124, 124, 125]:
        s = np.float32(2.0 ** e)
        for top in (4.0, 6.0, 7.0, 7.9999995):
            v = [np.float32(top)]
            for b in borders:
                v += [np.float32(b), np.nextafter(np.float32(b), np.float32(9)),
                      np.nextafter(np.float32(b), np.float32(0))]
            v += [np.float32(0), np.float32(-0.0), np.float32(1e-3)]
            v = np.array([a if abs(a) <= top else top for a in np.resize(v, 32)], np.float32)
            rows += [v * s, -v * s]
    _check_quantize(torch.from_numpy(np.stack(rows)))


def test_smallest_largest_and_zero_blocks():
    big = float(np.finfo(np.float32).max)
    x = torch.zeros(8, 96)
    x[1, 3] = 2.0 ** -149
    x[2] = 2.0 ** -127          # a tie at the smallest scale: goes to 0
    x[3] = 2.0 ** -127 * 1.5
    x[4] = big
    x[5, 32:64] = -big
    x[6, 5] = 2.0 ** -123
    x[7] = -0.0
    _check_quantize(x)
    _check_quantize(x.bfloat16())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_non_finite_blocks(dtype):
    x = normal(1, 5, 128, dtype=dtype)
    x[0, 3] = float("inf")
    x[1, 127] = float("nan")
    x[2, 32], x[2, 33] = float("-inf"), float("nan")
    x[3, 64:96] = float("nan")
    _check_quantize(x)


def test_every_code_under_every_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (251, 1))
    scales = np.arange(2, 253, dtype=np.uint8)[:, None].repeat(16, 1)
    scales[7, 3] = 255
    c, s = on_gpu((codes, scale_words(scales)))
    for dtype in (F32, BF16):
        got = B.moe_dequantize_mxfp4(c, s, dtype)
        assert np.array_equal(got.double().cpu().numpy(), values(codes, scales), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF16])
def test_more_rows_than_a_launch_takes(dtype):
    # rows of 128 words go in launches of 2^18; offsets pass 2^32 elements
    n, c = (1 << 18) + 3, 65536
    x = torch.zeros(n, c, dtype=dtype, device="cuda")
    at = torch.tensor([0, 1, 65535, 65536, (1 << 18) - 1, 1 << 18, n - 1])
    some = normal(5, at.numel(), c, dtype=dtype)
    x[at.cuda()] = some.cuda()
    codes, scales = B.moe_quantize_mxfp4(x)
    rc, rb = quantize_ref(some.double().numpy())
    assert np.array_equal(codes[at.cuda()].cpu().numpy(), rc)
    assert np.array_equal(scales[:, at.cuda()].cpu().numpy(), scale_words(rb))
    codes[at.cuda()] = 0
    scales[:, at.cuda()] = 2
    assert int(codes.max()) == 0 and int(scales.min()) == 2 and int(scales.max()) == 2
    x.fill_(1)
    codes[n - 1], scales[:, n - 1] = (torch.from_numpy(a).cuda()
                                      for a in (rc[-1], scale_words(rb)[:, -1]))
    B.moe_dequantize_mxfp4(codes, scales, x=x)
    assert np.array_equal(x[n - 1].double().cpu().numpy(), values(rc[-1:], rb[-1:])[0])
    x[n - 1] = 0
    assert not x.any()
    del x, codes, scales
    torch.cuda.empty_cache()


# ------------------------------------------------------------- products


def _weight(seed, e, rows, cols, mid=124):
    codes, scales = random_mxfp4(seed, e, rows, cols, mid=mid)
    return codes, scales, values(codes, scales)


def _left(seed, n, cols):
    codes, scales = random_mxfp4(seed, n, cols)
    return codes, scales, values(codes, scales)


def _gpu_weight(w):
    return B.Mxfp4Weight(*on_gpu(w[:2]))


def _gpu_left(x):
    return on_gpu((x[0], scale_words(x[1])))


def _product(w, x, offsets, left):
    """(out fp64 [slots][rows], its error before the last rounding); left[p]: x's row."""
    out = np.zeros((len(left), w[0].shape[1]))
    err = np.zeros_like(out)
    cols = w[2].shape[2]
    for e in range(w[0].shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b <= a:
            continue
        v = x[2][left[a:b]]
        out[a:b] = v @ w[2][e].T
        sums = np.abs(v) @ np.abs(w[2][e]).T
        unit = np.exp2(x[1][left[a:b]].min(axis=1).astype(np.float64) - 127)[:, None] * np.exp2(
            w[1][e].min(axis=1).astype(np.float64) - 127) / 4
        err[a:b] = np.where(sums < 2.0 ** 24 * unit, 0, (cols / 32 + 8) * 2.0 ** -20 * sums)
    return out, err


def _check(got, ref, err, what):
    bound = err + half_step(got.dtype) * (np.abs(ref) + err) + 2.0 ** -149
    assert_within(got, ref, bound, what)


def _check_swiglu(got, g, gerr, u, uerr, what):
    sig = np.exp(-np.logaddexp(0, -g))
    y = g * sig * u
    err = (2 * np.abs(g) + 10) * U32 * np.abs(y)
    err = err + 1.1 * gerr * np.abs(u) + uerr * np.abs(g * sig) + 2 * gerr * uerr
    # below -87 the sum 1 + e^-g or its reciprocal leaves fp32's normal numbers
    # and a value may be 0, as the header says: |g| e^g falls from 87 e^-87 =
    # 1.44e-36 on, so the value lost is below 1.5e-36 |u|
    _check(got, y, err + np.where(g < -86.9, 1.5e-36 * np.abs(u), 0), what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [
    (1, 1, 32, 0), (1, 4096, 4096, 0), (2, 33, 256, 1), (15, 16, 288, 0), (16, 17, 224, 0),
    (17, 1235, 2080, 0), (64, 64, 512, 0), (100, 300, 1056, 5), (129, 257, 544, 0),
    (257, 511, 1056, 0), (300, 128, 65536, 0), (513, 260, 3040, 0), (1030, 1025, 1312, 3)])
def test_dense_product(n, rows, cols, pad, dtype):
    print("case dense", n, rows, cols, pad, dtype, flush=True)
    _dense(n, rows, cols, pad, dtype)


def _dense(n, rows, cols, pad, dtype):
    w, u = _weight(n + rows, 1, rows, cols), _weight(n + rows + 1, 1, rows, cols)
    x = _left(7, n, cols)
    xd = _gpu_left(x)
    out = strided(torch.zeros(n, rows, dtype=dtype, device="cuda"), pad).fill_(float("nan"))
    assert B.moe_product_mxfp4(_gpu_weight(w), *xd, out=out) is out
    every = np.arange(n)
    a, aerr = _product(w, x, [0, n], every)
    _check(out, a, aerr, "out")
    got = B.moe_swiglu_mxfp4(_gpu_weight(w), _gpu_weight(u), *xd, out_dtype=dtype)
    _check_swiglu(got, a, aerr, *_product(u, x, [0, n], every), "swiglu")


# tokens, top_k, experts, experts used, share dropped, rows, cols
GROUPED = [
    (1, 1, 1, 1, 0.0, 16, 32),
    (1, 6, 256, 6, 0.0, 128, 1024),
    (7, 3, 5, 3, 0.3, 40, 352),
    (32, 6, 256, 120, 0.0, 64, 512),
    (33, 2, 1024, 60, 0.2, 19, 256),
    (100, 4, 16, 7, 0.1, 130, 544),
    (150, 8, 8, 8, 0.0, 260, 256),     # every expert takes every token
    (333, 3, 4, 3, 0.25, 100, 1280),
    (40, 2, 64, 2, 0.0, 256, 2048),    # two crowded experts, the rest empty
    (60, 4, 12, 12, 1.0, 48, 128),     # no slot has an expert
    (700, 2, 6, 5, 0.05, 320, 768),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,used,drop,rows,cols", GROUPED)
def test_grouped_products(n, k, e, used, drop, rows, cols, dtype):
    print("case grouped", n, k, e, used, drop, rows, cols, dtype, flush=True)
    g = group(make_ids(n, k, e, drop, used, seed=n + e), e)
    off, perm = g[1], g[2]
    total = int(off[-1])
    gd = on_gpu(g)
    gate, up = _weight(n, e, rows, cols), _weight(n + 1, e, rows, cols)
    gw, uw = _gpu_weight(gate), _gpu_weight(up)

    # gathered tokens, SwiGLU and plain
    x = _left(8, n, cols)
    xd = _gpu_left(x)
    left = perm // k
    a, b = _product(gate, x, off, left), _product(up, x, off, left)
    out = torch.full((n * k, rows), float("nan"), dtype=dtype, device="cuda")
    B.moe_swiglu_mxfp4(gw, uw, *xd, gd, top_k=k, out=out)
    _check_swiglu(out, *a, *b, "swiglu")
    assert not out[total:].any()
    out = B.moe_product_mxfp4(gw, *xd, gd, top_k=k, out_dtype=dtype)
    _check(out, *a, "gathered product")

    # rows in expert order; those past the last expert's hold anything
    x = _left(9, n * k, cols)
    x[1][total:] = 255
    x[2][total:] = 0
    out = torch.full((n * k, rows), float("nan"), dtype=dtype, device="cuda")
    B.moe_product_mxfp4(uw, *_gpu_left(x), gd, out=out)
    ref, err = _product(up, x, off, np.arange(n * k))
    _check(out, ref, err, "sorted product")
    assert not out[total:].any()


@pytest.mark.parametrize("n,rows,cols", [(1, 40, 4096), (300, 300, 4096), (40, 2000, 544)])
def test_scales_far_apart(n, rows, cols):
    # thirty binades of scales within a row: far from exact, within the bound
    # of the magnitudes' sum
    for seed, spread in ((1, 7), (2, 15)):
        c, s = random_mxfp4(seed, 1, rows, cols, spread=spread)
        w = c, s, values(c, s)
        c, s = random_mxfp4(seed + 10, n, cols, spread=spread)
        x = c, s, values(c, s)
        out = B.moe_product_mxfp4(_gpu_weight(w), *_gpu_left(x), out_dtype=F32)
        _check(out, *_product(w, x, [0, n], np.arange(n)), "out")


@pytest.mark.parametrize("n,rows", [(5, 70), (600, 520)])
def test_non_finite_blocks_stay_in_their_rows(n, rows):
    w, x = _weight(3, 1, rows, 320), _left(4, n, 320)
    x[1][3, 2] = 255
    x[0][3] = 0
    w[1][0, 11, 9] = 255
    out = B.moe_product_mxfp4(_gpu_weight(w), *_gpu_left(x), out_dtype=F32)
    assert torch.isnan(out[3]).all() and torch.isnan(out[:, 11]).all()
    ref, err = _product(w, x, [0, n], np.arange(n))
    keep = np.ix_(np.arange(n) != 3, np.arange(rows) != 11)
    _check(torch.from_numpy(out.cpu().numpy()[keep]), ref[keep], err[keep], "out")


FAR = [0.0, 0.5, 20, 60, 80, 86, 87, 87.5, 88, 88.5, 89, 90, 100, 104, 128, 300, 1000]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,e,rows,cols", [(36, 0, 40, 128), (36, 3, 33, 64), (1024, 0, 8192, 256),
                                           (700, 0, 6001, 512), (680, 4, 2048, 256),
                                           (4000, 1, 2048, 1024)])
def test_swiglu_of_far_gates_in_every_epilogue(n, e, rows, cols, dtype):
    # Gates around the places where exp(-g) leaves fp32 and its reciprocal the
    # normal numbers, and far past them: below -87 a value may be 0, where the
    # true one is at most 87 e^-87 |u|.  Half a step of a subnormal bf16 is
    # 2^-134, whatever its value.  A row's values sum to the gate exactly.
    gates = np.resize(np.array(FAR + [-v for v in FAR]), n)
    x = np.zeros((n, cols))
    for i, rest in enumerate(np.abs(gates)):
        # digits of 1 or 1.5 times a power of two, a block's second within a quarter of its first
        k, block = 0, 0.0
        while rest:
            top = 2.0 ** np.floor(np.log2(rest))
            if k % 32 == 1 and 4 * top >= block:
                k += 1
            else:
                k, block = -(-k // 32) * 32 + 1, top
            x[i, k - 1] = 1.5 * top if rest >= 1.5 * top else top
            rest -= x[i, k - 1]
    x *= np.sign(gates + (gates == 0))[:, None]
    xc, xs = quantize_ref(x)
    left = xc, xs, values(xc, xs)
    assert np.array_equal(left[2], x)
    ones = np.ones((max(e, 1), rows, cols))
    oc = np.full((max(e, 1), rows, cols // 2), 0x22, np.uint8)
    osc = np.full((max(e, 1), rows, cols // 32), 127, np.uint8)
    gate, up = (oc, osc, ones), _weight(6, max(e, 1), rows, cols)
    offsets = np.array([0, n]) if e == 0 else np.linspace(0, n, e + 1).astype(np.int32)
    filler = np.arange(n, dtype=np.int32)
    grouping = on_gpu((np.diff(offsets), offsets, filler, filler)) if e else None
    got = B.moe_swiglu_mxfp4(_gpu_weight(gate), _gpu_weight(up), *_gpu_left(left), grouping,
                             out_dtype=dtype)
    a, _ = _product(gate, left, offsets, np.arange(n))
    assert np.array_equal(a, gates[:, None].repeat(rows, 1))
    u, uerr = _product(up, left, offsets, np.arange(n))
    silu = a * np.exp(-np.logaddexp(0, -a))
    y = silu * u
    err = (2 * np.abs(a) + 10) * U32 * np.abs(y) + uerr * np.abs(silu)
    tol = err + half_step(dtype) * (np.abs(y) + err) + 2.0 ** -149
    tol += 2.0 ** -134 if dtype == BF16 else 0
    assert_within(got, y, tol + np.where(a < -86.9, 1.5e-36 * np.abs(u), 0), "far gates")


def test_a_layer_of_the_calls_together():
    # norm, route, gate and up, round, down, combine, against the same steps on
    # the values that the rounded rows stand for
    n, k, e, hidden, inter = 70, 3, 8, 256, 160
    x, res = normal(1, n, hidden, dtype=BF16).cuda(), normal(2, n, hidden, dtype=BF16).cuda()
    w = (1 + 0.2 * normal(3, hidden)).cuda()
    gate, up = _weight(4, e, inter, hidden, mid=120), _weight(5, e, inter, hidden, mid=120)
    down = _weight(6, e, hidden, inter, mid=120)
    logits = normal(7, n, e).cuda()
    codes, scales, total = B.moe_rmsnorm_mxfp4(x, w, residual=res)
    ids, tw, grouping = B.moe_route_group(logits, k)
    h = B.moe_swiglu_mxfp4(_gpu_weight(gate), _gpu_weight(up), codes, scales, grouping, top_k=k,
                           out_dtype=F32)
    hc, hs = B.moe_quantize_mxfp4(h)
    rows = B.moe_product_mxfp4(_gpu_weight(down), hc, hs, grouping, out_dtype=F32)
    y = B.moe_combine(rows, tw, grouping, base=total)
    # each step on the one before it
    xv = values(codes.cpu().numpy(), B.mxfp4_scale_rows(scales, hidden).cpu().numpy())
    xl = codes.cpu().numpy(), B.mxfp4_scale_rows(scales, hidden).cpu().numpy(), xv
    off, perm = (grouping[i].cpu().numpy() for i in (1, 2))
    left = perm // k
    a, b = _product(gate, xl, off, left), _product(up, xl, off, left)
    _check_swiglu(h, *a, *b, "h")
    rc, rb = quantize_ref(h.double().cpu().numpy())
    assert np.array_equal(hc.cpu().numpy(), rc)
    hl = rc, rb, values(rc, rb)
    ref, err = _product(down, hl, off, np.arange(n * k))
    _check(rows, ref, err, "rows")
    inv = grouping[3].cpu().numpy().reshape(n, k)
    tw64 = tw.double().cpu().numpy()
    want = total.double().cpu().numpy() + sum(tw64[:, i:i + 1] * ref[inv[:, i]] for i in range(k))
    mags = sum(tw64[:, i:i + 1] * (np.abs(ref) + err)[inv[:, i]] for i in range(k)) + np.abs(
        total.double().cpu().numpy())
    errs = sum(tw64[:, i:i + 1] * err[inv[:, i]] for i in range(k)) + (k + 2) * U32 * mags
    assert_within(y, want, errs + half_step(BF16) * (np.abs(want) + errs), "y")


def test_two_streams_at_once():
    # the same weights and left operands on two streams, in turns without a wait
    n, k, e, rows, cols = 64, 4, 16, 320, 1056
    g = on_gpu(group(make_ids(n, k, e, 0.1, seed=2), e))
    gate, up = (_gpu_weight(_weight(i, e, rows, cols)) for i in (1, 2))
    x = _gpu_left(_left(3, n, cols))
    want = B.moe_swiglu_mxfp4(gate, up, *x, g, top_k=k), B.moe_product_mxfp4(gate, *x, g, top_k=k)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        got += [(B.moe_swiglu_mxfp4(gate, up, *x, g, top_k=k, stream=s),
                 B.moe_product_mxfp4(gate, *x, g, top_k=k, stream=s)) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))


def test_no_slots():
    w = _gpu_weight(_weight(1, 4, 32, 64))
    g = on_gpu(group(make_ids(0, 2, 4), 4))
    codes, scales = B.moe_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (1, 0, 16)
    assert B.moe_product_mxfp4(w, codes, scales, g, top_k=2).shape == (0, 32)
    assert B.moe_dequantize_mxfp4(codes, scales).shape == (0, 64)


def test_left_rows_past_32_bit_offsets():
    # 70000 rows of 32768 bytes of codes: the last lie past 2^31; some are looked at
    n, c = 70000, 65536
    codes = torch.zeros((n, c // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((c // 512, n, 16), 127, dtype=torch.uint8, device="cuda")
    at = np.array([0, 1, 65535, 65536, 65537, 69999])
    some = _left(5, 6, c)
    codes[torch.from_numpy(at).cuda()] = torch.from_numpy(some[0]).cuda()
    scales[:, torch.from_numpy(at).cuda()] = torch.from_numpy(scale_words(some[1])).cuda()
    w = _weight(6, 1, 16, c)
    out = B.moe_product_mxfp4(_gpu_weight(w), codes, scales, out_dtype=F32)
    _check(out[torch.from_numpy(at).cuda()], *_product(w, some, [0, 6], np.arange(6)), "out")
    rest = torch.ones(n, dtype=torch.bool)
    rest[torch.from_numpy(at)] = False
    assert not out[rest.cuda()].any()
    del codes, scales, out
    torch.cuda.empty_cache()


def test_results_repeat_on_another_stream_and_in_a_graph():
    n, k, e, rows, cols = 48, 4, 16, 192, 512
    g = on_gpu(group(make_ids(n, k, e, 0.1, seed=2), e))
    gate, up = (_gpu_weight(_weight(i, e, rows, cols)) for i in (1, 2))
    x = normal(3, n, cols, dtype=BF16).cuda()

    def passes(stream=None):
        q, s = B.moe_quantize_mxfp4(x, stream=stream)
        h = B.moe_swiglu_mxfp4(gate, up, q, s, g, top_k=k, stream=stream)
        y = B.moe_product_mxfp4(gate, q, s, g, top_k=k, out_dtype=F32, stream=stream)
        return q, s, h, y, B.moe_dequantize_mxfp4(q, s, stream=stream)

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


def test_products_on_groupings_of_moe_group_with_dropped_slots():
    # moe_group writes perm up to the last expert's row only
    n, k, e, rows, cols = 90, 4, 16, 48, 416
    ids = make_ids(n, k, e, 0.3, seed=11)
    counts, off, perm, inv = group(ids, e)
    total = int(off[-1])
    g = [torch.full((m,), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
         for m in (e, e + 1, n * k, n * k)]
    grouping = B.moe_group(torch.from_numpy(ids).cuda(), e, out=tuple(g))
    gate, up, x = _weight(1, e, rows, cols), _weight(2, e, rows, cols), _left(3, n, cols)
    a, b = _product(gate, x, off, perm // k), _product(up, x, off, perm // k)
    out = torch.full((n * k, rows), float("nan"), dtype=F32, device="cuda")
    B.moe_product_mxfp4(_gpu_weight(gate), *_gpu_left(x), grouping, top_k=k, out=out)
    _check(out, *a, "product")
    assert not out[total:].any()
    out.fill_(float("nan"))
    B.moe_swiglu_mxfp4(_gpu_weight(gate), _gpu_weight(up), *_gpu_left(x), grouping, top_k=k,
                       out=out)
    _check_swiglu(out, *a, *b, "swiglu")
    assert not out[total:].any()


def test_weights_take_scale_rows_of_any_width():
    w, x = _weight(1, 2, 40, 96), _left(2, 6, 96)
    wide = np.full((2, 40, 16), 200, np.uint8)
    wide[..., :3] = w[1]
    g = on_gpu((np.array([3, 3], np.int32), np.array([0, 3, 6], np.int32),
                np.arange(6, dtype=np.int32), np.arange(6, dtype=np.int32)))
    want = B.moe_product_mxfp4(_gpu_weight(w), *_gpu_left(x), g)
    got = B.moe_product_mxfp4(B.Mxfp4Weight(*on_gpu((w[0], wide))), *_gpu_left(x), g)
    assert torch.equal(got, want)


def test_refusals_on_the_gpu():
    # returned before anything is enqueued
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(B.MoeError) as err:
        B.moe_quantize_mxfp4(x[:, :48].contiguous())
    assert err.value.status == B.MOE_ERR_UNSUPPORTED and "moe_quantize_mxfp4" in str(err.value)
    codes, scales = B.moe_quantize_mxfp4(x)
    g = on_gpu(group(make_ids(4, 2, 8), 8))
    w = _gpu_weight(_weight(1, 8, 32, 64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        B.moe_product_mxfp4(w, codes, scales, g, top_k=2, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="scales must be"):
        B.moe_product_mxfp4(w, codes, scales[:, :3], g, top_k=2)
    with pytest.raises(ValueError, match="codes must be"):
        B.moe_product_mxfp4(w, codes[:, :16].contiguous(), scales, g, top_k=2)
    with pytest.raises(B.MoeError):
        B.moe_product_mxfp4(w, codes, scales)  # several matrices, no grouping
    with pytest.raises(B.MoeError):
        B.moe_swiglu_mxfp4(w, _gpu_weight(_weight(1, 8, 48, 64)), codes, scales, g, top_k=2)
    torch.cuda.synchronize()


