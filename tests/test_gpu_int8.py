"""Rounding to int8 and the int8 products against 64-bit references.

Bounds: q and the scales are exact (the scale is one fp32 division).  The
int32 sum is exact; turned to fp32 and multiplied by two scales it is off by
three half-steps of fp32, then half a step of the output's type.  SwiGLU's
quotient g / (1 + e^-g) has condition number 1 + |g| in g; the exponential
(4 half-steps), the sum, the quotient and the last product come on top, and u
brings its own three."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from rows_testlib import (U32, assert_within, group, half_step, int8_weight, make_ids, normal,
                          on_gpu, product_ref, quantize_ref, strided)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,c,pad", [(1, 16, 0), (1, 4096, 0), (3, 48, 1), (17, 2064, 7),
                                     (130, 1024, 0), (5, 65536, 0), (2, 8208, 3),
                                     (700, 4096, 0)])
def test_quantize_is_exact(n, c, pad, dtype):
    print("case quantize", n, c, pad, dtype, flush=True)
    x = normal(n + c, n, c)
    x[:, ::97] *= 12
    x = x.to(dtype)
    # exact halves and values right beside them: fractions (m + 1/2) / 127 of
    # the largest value, which is a multiple of 127 here
    x[0] = 0
    halves = torch.arange(0, min(c - 1, 127), dtype=torch.float32) + 0.5
    x[0, 1:1 + halves.numel()] = halves * 2
    x[0, 0] = 254
    q, s = B.moe_quantize_int8(strided(x.cuda(), pad))
    rq, rs = quantize_ref(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs)


def test_quantize_borders_in_fp32():
    # values one fp32 step around every border of a row whose largest value
    # makes the borders inexact
    for top in (1.0, 3.1415927, 1e-20, 7e30, 3e-39, 1.0000001):
        a = np.float32(top)
        border = ((np.arange(-127, 127) + 0.5) / 127 * np.float64(a)).astype(np.float32)
        v = np.concatenate([[a], border, np.nextafter(border, np.float32(np.inf)),
                            np.nextafter(border, np.float32(-np.inf))]).astype(np.float32)
        v = np.clip(np.resize(v, 768), -a, a)
        q, s = B.moe_quantize_int8(torch.from_numpy(v).reshape(1, -1).cuda())
        rq, rs = quantize_ref(v.reshape(1, -1))
        assert np.array_equal(q.cpu().numpy(), rq), top
        assert np.array_equal(s.cpu().numpy(), rs), top


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_zero_and_non_finite_rows(dtype):
    x = normal(1, 6, 64, dtype=dtype)
    x[1] = 0.0
    x[2] = -0.0
    x[3, 5] = float("inf")
    x[4, 63] = float("nan")
    x[5, 0] = float("-inf")
    x[5, 1] = float("nan")
    q, s = (t.cpu().numpy() for t in B.moe_quantize_int8(x.cuda()))
    rq, rs = quantize_ref(x[:3].double().numpy())
    assert np.array_equal(q[:3], rq) and np.array_equal(s[:3], rs)
    assert not q[1:].any()
    assert np.array_equal(s[1:3], np.zeros(2, np.float32)) and np.isnan(s[3:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_more_rows_than_a_launch_takes(dtype):
    # rows go in launches of 2^22; the reference in 64 bits on the GPU
    n, c = (1 << 22) + 5, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, c, generator=g, device="cuda").to(dtype)
    for r in ((1 << 22) - 1, 1 << 22, n - 1):
        x[r] *= 100
    x[(1 << 22) + 1] = 0
    x[(1 << 22) + 2, 3] = float("inf")
    q = torch.full((n, c), 77, dtype=torch.int8, device="cuda")
    s = torch.full((n,), -1.0, device="cuda")
    B.moe_quantize_int8(x, q=q, scale=s)
    bad = (1 << 22) + 2
    assert bool(s[bad].isnan()) and not q[bad].any()
    x[bad] = 0
    a = x.double().abs().amax(1, keepdim=True)
    ref = torch.round(x.double() * 127 / a.clamp_min(1e-300)).to(torch.int8)
    assert torch.equal(q, ref)
    s[bad] = 0
    # from 64 bits: torch takes an fp32 tensor over a number by its reciprocal
    assert torch.equal(s, (a[:, 0] / 127).float())


def _bound(ref, dtype, steps):
    err = steps * U32 * np.abs(ref) * (1 + 2.0 ** -20)
    return err + half_step(dtype) * (np.abs(ref) + err) + 2.0 ** -149


def _swiglu(g, u):
    y = g / (1 + np.exp(-g)) * u
    return y, 3 * (1 + np.abs(g)) + 4 + 1 + 1 + 3 + 1


def _left(n, cols, seed):
    rng = np.random.default_rng(seed)
    return (rng.integers(-128, 128, (n, cols), dtype=np.int8),
            rng.uniform(0.01, 0.03, n).astype(np.float32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [
    (1, 1, 16, 0), (1, 4096, 4096, 0), (2, 33, 128, 1), (15, 16, 144, 0), (16, 17, 112, 0),
    (17, 1235, 2064, 0), (64, 64, 512, 0), (100, 300, 1040, 5), (129, 257, 256, 0),
    (257, 511, 528, 0), (300, 128, 65536, 0), (513, 260, 1536, 0), (1030, 1025, 640, 3)])
def test_dense_product(n, rows, cols, pad, dtype):
    print("case dense", n, rows, cols, pad, dtype, flush=True)
    wq, ws = int8_weight(n + rows, 1, rows, cols)
    q, s = _left(n, cols, 7)
    w = B.Int8Weight(torch.from_numpy(wq[0]).cuda(), torch.from_numpy(ws[0]).cuda())
    out = strided(torch.zeros(n, rows, dtype=dtype, device="cuda"), pad).fill_(float("nan"))
    got = B.moe_product_int8(w, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), out=out)
    assert got is out
    ref = product_ref(wq, ws, q, s, [0, n], np.arange(n))
    assert_within(out, ref, _bound(ref, dtype, 3), "out")
    up, us = int8_weight(n + rows + 1, 1, rows, cols)
    u = B.Int8Weight(torch.from_numpy(up[0]).cuda(), torch.from_numpy(us[0]).cuda())
    got = B.moe_swiglu_int8(w, u, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(),
                            out_dtype=dtype)
    y, steps = _swiglu(ref, product_ref(up, us, q, s, [0, n], np.arange(n)))
    assert_within(got, y, _bound(y, dtype, steps), "swiglu")


# tokens, top_k, experts, experts used, share dropped, rows, cols
GROUPED = [
    (1, 1, 1, 1, 0.0, 16, 16),
    (1, 6, 256, 6, 0.0, 128, 512),
    (7, 3, 5, 3, 0.3, 40, 176),
    (32, 6, 256, 120, 0.0, 64, 256),
    (33, 2, 1024, 60, 0.2, 19, 128),
    (100, 4, 16, 7, 0.1, 130, 272),
    (150, 8, 8, 8, 0.0, 260, 128),     # every expert takes every token
    (333, 3, 4, 3, 0.25, 100, 640),
    (40, 2, 64, 2, 0.0, 256, 1024),    # two crowded experts, the rest empty
    (60, 4, 12, 12, 1.0, 48, 64),      # no slot has an expert
    (700, 2, 6, 5, 0.05, 320, 384),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,used,drop,rows,cols", GROUPED)
def test_grouped_products(n, k, e, used, drop, rows, cols, dtype):
    print("case grouped", n, k, e, used, drop, rows, cols, dtype, flush=True)
    ids = make_ids(n, k, e, drop, used, seed=n + e)
    g = group(ids, e)
    off, perm = g[1], g[2]
    total = int(off[-1])
    gd = on_gpu(g)
    (gq, gs), (uq, us) = int8_weight(n, e, rows, cols), int8_weight(n + 1, e, rows, cols)
    gate, up = (B.Int8Weight(*on_gpu(w)) for w in ((gq, gs), (uq, us)))

    # gathered tokens, SwiGLU and plain
    q, s = _left(n, cols, 8)
    qd, sd = on_gpu((q, s))
    left = perm // k
    a = product_ref(gq, gs, q, s, off, left)
    b = product_ref(uq, us, q, s, off, left)
    out = torch.full((n * k, rows), float("nan"), dtype=dtype, device="cuda")
    B.moe_swiglu_int8(gate, up, qd, sd, gd, top_k=k, out=out)
    y, steps = _swiglu(a, b)
    assert_within(out, y, _bound(y, dtype, steps), "swiglu")
    assert not out[total:].any()
    out = B.moe_product_int8(gate, qd, sd, gd, top_k=k, out_dtype=dtype)
    assert_within(out, a, _bound(a, dtype, 3), "gathered product")

    # rows in expert order; those past the last expert's hold anything
    q, s = _left(n * k, cols, 9)
    s[total:] = np.nan
    qd, sd = on_gpu((q, s))
    out = torch.full((n * k, rows), float("nan"), dtype=dtype, device="cuda")
    B.moe_product_int8(up, qd, sd, gd, out=out)
    ref = product_ref(uq, us, q, s, off, np.arange(n * k))
    assert_within(out, ref, _bound(ref, dtype, 3), "sorted product")
    assert not out[total:].any()


def test_extreme_values_sum_exactly():
    # 65536 products of -128 * -128 and of -128 * 127: 2^30 and its like in int32
    c = 65536
    q = np.full((2, c), -128, np.int8)
    w = np.stack([np.full(c, -128, np.int8), np.full(c, 127, np.int8)])
    out = B.moe_product_int8(B.Int8Weight(*on_gpu((w, np.ones(2, np.float32)))),
                             *on_gpu((q, np.ones(2, np.float32))), out_dtype=F32)
    assert out.cpu().tolist() == [[float(2 ** 30), float(-128 * 127 * c)]] * 2


def test_non_finite_scales_stay_in_their_rows():
    wq, ws = int8_weight(3, 1, 70, 128)
    q, s = _left(40, 128, 4)
    s[5] = np.nan
    q[5] = 0
    out = B.moe_product_int8(B.Int8Weight(*on_gpu((wq, ws))), *on_gpu((q, s)), out_dtype=F32)
    assert torch.isnan(out[5]).all()
    keep = np.arange(40) != 5
    ref = product_ref(wq, ws, q, s, [0, 40], np.arange(40))[keep]
    assert_within(out[torch.from_numpy(keep).cuda()], ref, _bound(ref, F32, 3), "out")


def test_swiglu_of_far_gates():
    # gates of hundreds either way: SiLU is g or vanishes
    c, rows = 64, 32
    gq = np.full((1, rows, c), 1, np.int8)
    q = np.stack([np.full(c, v, np.int8) for v in (-127, -20, -1, 0, 1, 20, 127)])
    s = np.full(7, 0.25, np.float32)
    one = np.ones((1, rows), np.float32)
    w = B.Int8Weight(*on_gpu((gq, one)))
    out = B.moe_swiglu_int8(w, w, *on_gpu((q, s)), out_dtype=F32)
    a = product_ref(gq, one, q, s, [0, 7], np.arange(7))
    y = a * np.exp(-np.logaddexp(0, -a)) * a
    assert_within(out, y, _bound(y, F32, 3 * (1 + np.abs(a)) + 10) + 1e-30, "far gates")


FAR = [0.0, 0.5, 20, 60, 80, 86, 87, 87.5, 88, 88.5, 88.8, 89, 90, 100, 104, 127, 300, 1000]


# rows and channels of the kernel for few rows and of tiled ones, 16-byte
# bf16 stores among them, dense (experts 0) and grouped
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,e,rows,cols,tiled", [
    (36, 0, 40, 64, False), (36, 3, 33, 64, False), (1024, 0, 8192, 128, True),
    (700, 0, 6001, 512, True), (680, 4, 2048, 256, True), (4000, 1, 2048, 1024, True)])
def test_swiglu_of_far_gates_in_every_epilogue(n, e, rows, cols, tiled, dtype):
    # Gates around the places where exp(-g) leaves fp32 and its reciprocal the
    # normal numbers, and far past them.  The hardware's exponential and
    # reciprocal add 2 |g| half-steps of fp32 to the bound above; below -87 a
    # value may be 0, where the true one is at most 87 e^-87 |u|.  Half a step
    # of a subnormal bf16 is 2^-134, whatever its value.
    assert (B.moe_int8_form(e or 1, rows, cols, n, e > 0, True)[2] > 0) == tiled
    gates = np.resize(np.array(FAR + [-v for v in FAR], np.float32), n)
    ones = np.ones((e or 1, rows, cols), np.int8)
    uq, us = int8_weight(6, e or 1, rows, cols)
    q = np.where(gates < 0, -1, 1).astype(np.int8)[:, None].repeat(cols, 1)
    s = np.abs(gates) / np.float32(cols)
    unit = np.ones((e or 1, rows), np.float32)
    offsets = np.array([0, n]) if e == 0 else np.linspace(0, n, e + 1).astype(np.int32)
    filler = np.arange(n, dtype=np.int32)
    grouping = on_gpu((np.diff(offsets), offsets, filler, filler)) if e else None
    got = B.moe_swiglu_int8(*(B.Int8Weight(*on_gpu(w)) for w in ((ones, unit), (uq, us))),
                            *on_gpu((q, s)), grouping, out_dtype=dtype)
    a = product_ref(ones, unit, q, s, offsets, np.arange(n))
    u = product_ref(uq, us, q, s, offsets, np.arange(n))
    y = a * np.exp(-np.logaddexp(0, -a)) * u
    tol = _bound(y, dtype, 3 * (1 + np.abs(a)) + 10 + 2 * np.abs(a))
    tol += 2.0 ** -134 if dtype == BF16 else 0
    assert_within(got, y, tol + np.where(a < -86.9, 1.5e-36 * np.abs(u), 0), "far gates")


def test_no_slots():
    w = B.Int8Weight(*on_gpu(int8_weight(1, 4, 32, 64)))
    g = on_gpu(group(make_ids(0, 2, 4), 4))
    q, s = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    assert B.moe_product_int8(w, q, s, g, top_k=2).shape == (0, 32)
    q, s = B.moe_quantize_int8(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


def test_left_rows_past_32_bit_offsets():
    # 40000 rows of 65536 bytes: the last lie past 2^31; only some rows are looked at
    n, c = 40000, 65536
    q = torch.zeros((n, c), dtype=torch.int8, device="cuda")
    look = torch.tensor([0, 1, 32767, 32768, 32769, 39999])
    vals, _ = _left(6, c, 5)
    q[look.cuda()] = torch.from_numpy(vals).cuda()
    wq, ws = int8_weight(6, 1, 16, c)
    out = B.moe_product_int8(B.Int8Weight(*on_gpu((wq, ws))), q,
                             torch.ones(n, device="cuda"), out_dtype=F32)
    ref = product_ref(wq, ws, vals, np.ones(6, np.float32), [0, 6], np.arange(6))
    assert_within(out[look.cuda()], ref, _bound(ref, F32, 3), "out")
    look2 = torch.ones(n, dtype=torch.bool)
    look2[look] = False
    assert not out[look2.cuda()].any()
    del q, out
    torch.cuda.empty_cache()


def test_results_repeat_on_another_stream_and_in_a_graph():
    n, k, e, rows, cols = 48, 4, 16, 192, 512
    g = on_gpu(group(make_ids(n, k, e, 0.1, seed=2), e))
    gate, up = (B.Int8Weight(*on_gpu(int8_weight(i, e, rows, cols))) for i in (1, 2))
    x = normal(3, n, cols, dtype=BF16).cuda()

    def passes(stream=None):
        q, s = B.moe_quantize_int8(x, stream=stream)
        h = B.moe_swiglu_int8(gate, up, q, s, g, top_k=k, stream=stream)
        y = B.moe_product_int8(gate, q, s, g, top_k=k, out_dtype=F32, stream=stream)
        return q, s, h, y

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


def _dense(n, rows, cols, pad, dtype):
    wq, ws = int8_weight(n + rows, 1, rows, cols)
    uq, us = int8_weight(n + rows + 1, 1, rows, cols)
    q, s = _left(n, cols, 7)
    w, u = B.Int8Weight(*on_gpu((wq, ws))), B.Int8Weight(*on_gpu((uq, us)))
    qd, sd = on_gpu((q, s))
    out = strided(torch.zeros(n, rows, dtype=dtype, device="cuda"), pad).fill_(float("nan"))
    B.moe_product_int8(w, qd, sd, out=out)
    ref = product_ref(wq, ws, q, s, [0, n], np.arange(n))
    assert_within(out, ref, _bound(ref, dtype, 3), "out")
    got = B.moe_swiglu_int8(w, u, qd, sd, out_dtype=dtype)
    y, steps = _swiglu(ref, product_ref(uq, us, q, s, [0, n], np.arange(n)))
    assert_within(got, y, _bound(y, dtype, steps), "swiglu")


# sizes of the tiled kernels: rows of every tile height, ragged in each
# dimension, reductions of less than one step to several
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [
    (1030, 8200, 176, 3), (1024, 8192, 128, 0), (600, 8500, 64, 0), (2000, 4099, 1296, 1),
    (200, 16500, 144, 0), (100, 20011, 272, 1), (129, 18000, 16, 0), (100, 19000, 640, 0),
    (33, 45001, 256, 0), (48, 45000, 400, 0)])
def test_dense_product_of_many_tiles(n, rows, cols, pad, dtype):
    print("case dense tiles", n, rows, cols, pad, dtype, flush=True)
    _dense(n, rows, cols, pad, dtype)


# tokens, top_k, experts, experts used, share dropped, rows, cols
GROUPED_TILES = [
    (50, 4, 64, 40, 0.2, 2000, 144),
    (50, 4, 64, 40, 0.0, 2048, 16),
    (64, 6, 256, 120, 0.1, 1027, 400),
    (500, 2, 1024, 900, 0.1, 260, 256),
    (300, 4, 40, 33, 0.1, 1500, 272),
    (300, 4, 40, 4, 0.0, 1500, 128),
    (400, 6, 24, 20, 0.2, 1300, 144),
    (400, 6, 24, 24, 0.0, 1313, 528),
    (700, 3, 5, 4, 0.1, 1100, 208),
    (2600, 2, 6, 6, 0.3, 600, 640),
    (900, 4, 12, 12, 1.0, 1024, 64),   # no slot has an expert
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,used,drop,rows,cols", GROUPED_TILES)
def test_grouped_products_of_many_tiles(n, k, e, used, drop, rows, cols, dtype):
    test_grouped_products(n, k, e, used, drop, rows, cols, dtype)


# sizes at which the other tile shapes are chosen: 256 x 256, 128 x 256, 128 x
# 128 and 64 x 64, plain and with SwiGLU
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [
    (4339, 1870, 192, 1), (3811, 4127, 192, 0), (2335, 1697, 272, 0), (1236, 1649, 1184, 3),
    (4170, 771, 16, 0), (4365, 227, 16, 0), (514, 3585, 272, 1), (132, 6955, 16, 0)])
def test_dense_product_of_every_tile_shape(n, rows, cols, pad, dtype):
    print("case dense shapes", n, rows, cols, pad, dtype, flush=True)
    _dense(n, rows, cols, pad, dtype)


# tokens, top_k, experts, experts used, share dropped, rows, cols
GROUPED_FORMS = [
    (1011, 4, 5, 5, 0.1, 450, 1696),
    (201, 2, 8, 7, 0.2, 3972, 288),
    (756, 6, 64, 60, 0.1, 538, 272),
    (615, 6, 150, 140, 0.2, 187, 16),
    (832, 2, 40, 33, 0.0, 669, 320),
    (143, 5, 1024, 500, 0.1, 55, 16),
    (1029, 3, 150, 120, 0.1, 162, 592),
    (7171, 1, 1, 1, 0.1, 1047, 160),
    (7170, 1, 1, 1, 0.05, 2276, 176),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,used,drop,rows,cols", GROUPED_FORMS)
def test_grouped_products_of_every_tile_shape(n, k, e, used, drop, rows, cols, dtype):
    test_grouped_products(n, k, e, used, drop, rows, cols, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", [(4061, 2111, 3184, 0), (4061, 1055, 3184, 1),
                                             (67, 5366, 16, 0), (65, 6587, 16, 3)])
def test_dense_product_of_more_tile_shapes(n, rows, cols, pad, dtype):
    print("case dense more shapes", n, rows, cols, pad, dtype, flush=True)
    _dense(n, rows, cols, pad, dtype)


# Several tiles for every persistent workgroup, so that the rings of steps and
# of scales run on across tiles: every tile shape, plain and with SwiGLU, with
# reductions of one step where a shape is chosen for such, and of several
# (test_ops_host.py checks which shapes these reach).  The 64-bit references
# are taken on the GPU.
SEVERAL_TILES = [
    (65, 17021, 16, 0), (67, 33120, 16, 3), (16561, 200, 16, 0), (14482, 257, 144, 1),
    (64, 37142, 880, 0), (16500, 272, 16, 0), (16482, 277, 144, 0), (195, 35940, 16, 0),
    (18731, 386, 144, 0), (18287, 516, 16, 1), (36564, 258, 1424, 0), (22016, 293, 1584, 0),
    (38470, 260, 272, 0), (36081, 273, 800, 5), (132, 38743, 816, 0), (24350, 779, 2256, 0),
    (23415, 1695, 2192, 1),
]
# slots, experts, share without an expert, rows, cols
GROUPED_SEVERAL_TILES = [
    (240, 222, 0.0, 263, 16), (480, 283, 0.0, 278, 16), (1500, 291, 0.05, 267, 144),
    (290, 188, 0.0, 560, 784), (4500, 145, 0.0, 275, 16), (4300, 253, 0.02, 290, 16),
    (3900, 241, 0.0, 296, 896), (7600, 285, 0.0, 326, 16), (2400, 121, 0.0, 1040, 864),
    (11300, 29, 0.0, 259, 144), (23600, 27, 0.01, 333, 16), (15200, 94, 0.0, 258, 2720),
    (2700, 57, 0.0, 1264, 288), (24200, 151, 0.02, 290, 272), (20700, 154, 0.0, 274, 848),
    (9900, 37, 0.03, 1056, 3296), (3300, 12, 0.0, 7007, 3088),
]


def several_tiles_offsets(slots, e, share, seed):
    """offsets int32 [e + 1]; slots' experts are uniform, some slots have none."""
    rng = np.random.default_rng(seed)
    counts = np.bincount(rng.integers(0, e, slots - int(slots * share)), minlength=e)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _on_gpu_product(w, q, s, offsets):
    out = torch.zeros(q.shape[0], w.rows, dtype=torch.float64, device="cuda")
    for e in range(w.q.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            acc = q[a:b].double() @ w.q[e].double().t().contiguous()
            out[a:b] = acc * s[a:b, None].double() * w.scale[e].double()
    return out


def _gpu_within(got, ref, steps, what):
    err = steps * U32 * ref.abs() * (1 + 2.0 ** -20)
    bound = err + half_step(got.dtype) * (ref.abs() + err) + 2.0 ** -149
    over = (got.double() - ref).abs() - bound
    assert bool(torch.isfinite(got).all()), what
    worst = int(over.argmax())
    assert float(over.view(-1)[worst]) <= 0, (what, divmod(worst, ref.shape[1]))


def _several_tiles(slots, e, rows, cols, pad, dtype, offsets, grouping, top_k=0):
    g = torch.Generator(device="cuda").manual_seed(slots + rows)

    def ints(*shape):
        return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    w, u = (B.Int8Weight(ints(e, rows, cols), uniform(0.5, 2.0, e, rows) / (74 * cols ** 0.5))
            for _ in range(2))
    q, s = ints(slots, cols), uniform(0.01, 0.03, slots)
    out = strided(torch.zeros(slots, rows, dtype=dtype, device="cuda"), pad).fill_(float("nan"))
    B.moe_product_int8(w, q, s, grouping, out=out)
    a = _on_gpu_product(w, q, s, offsets)
    _gpu_within(out, a, 3, "out")
    out.fill_(float("nan"))
    B.moe_swiglu_int8(w, u, q, s, grouping, out=out)
    y = a / (1 + torch.exp(-a)) * _on_gpu_product(u, q, s, offsets)
    _gpu_within(out, y, 3 * (1 + a.abs()) + 10, "swiglu")
    assert not out[int(offsets[-1]):].any()
    if top_k:  # every row's token gathered
        live = int(offsets[-1])
        tokens = (grouping[2][:live] // top_k).long()
        qs = torch.zeros_like(q), torch.zeros_like(s)
        q, s = q[:slots // top_k], s[:slots // top_k]
        qs[0][:live], qs[1][:live] = q[tokens], s[tokens]
        out.fill_(float("nan"))
        B.moe_product_int8(w, q, s, grouping, top_k=top_k, out=out)
        _gpu_within(out, _on_gpu_product(w, *qs, offsets), 3, "gathered")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols,pad", SEVERAL_TILES)
def test_dense_product_of_several_tiles_a_workgroup(n, rows, cols, pad, dtype):
    print("case dense several", n, rows, cols, pad, dtype, flush=True)
    _several_tiles(n, 1, rows, cols, pad, dtype, [0, n], None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("slots,e,share,rows,cols", GROUPED_SEVERAL_TILES)
def test_grouped_product_of_several_tiles_a_workgroup(slots, e, share, rows, cols, dtype):
    print("case grouped several", slots, e, share, rows, cols, dtype, flush=True)
    offsets = several_tiles_offsets(slots, e, share, seed=slots + e)
    perm = np.random.default_rng(slots).permutation(slots).astype(np.int32)
    perm[offsets[-1]:] = -77  # as moe_group leaves it: anything
    grouping = on_gpu((np.diff(offsets), offsets, perm, perm))
    _several_tiles(slots, e, rows, cols, 0, dtype, offsets, grouping, top_k=2)


def test_products_on_groupings_of_moe_group_with_dropped_slots():
    # moe_group writes perm up to the last expert's row only
    n, k, e, rows, cols = 90, 4, 16, 48, 208
    ids = make_ids(n, k, e, 0.3, seed=11)
    counts, off, perm, inv = group(ids, e)
    total = int(off[-1])
    g = [torch.full((m,), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
         for m in (e, e + 1, n * k, n * k)]
    grouping = B.moe_group(torch.from_numpy(ids).cuda(), e, out=tuple(g))
    assert np.array_equal(grouping[1].cpu().numpy(), off) and 0 < total < n * k
    (gq, gs), (uq, us) = int8_weight(1, e, rows, cols), int8_weight(2, e, rows, cols)
    gate, up = (B.Int8Weight(*on_gpu(w)) for w in ((gq, gs), (uq, us)))
    q, s = _left(n, cols, 3)
    left = perm // k
    a, b = (product_ref(*w, q, s, off, left) for w in ((gq, gs), (uq, us)))
    out = torch.full((n * k, rows), float("nan"), dtype=F32, device="cuda")
    B.moe_product_int8(gate, *on_gpu((q, s)), grouping, top_k=k, out=out)
    assert_within(out, a, _bound(a, F32, 3), "product")
    assert not out[total:].any()
    out.fill_(float("nan"))
    B.moe_swiglu_int8(gate, up, *on_gpu((q, s)), grouping, top_k=k, out=out)
    y, steps = _swiglu(a, b)
    assert_within(out, y, _bound(y, F32, steps), "swiglu")
    assert not out[total:].any()


def test_refusals_on_the_gpu():
    # returned before anything is enqueued
    x = torch.zeros(4, 64, device="cuda")
    g = on_gpu(group(make_ids(4, 2, 8), 8))
    with pytest.raises(B.MoeError) as e:
        B.moe_quantize_int8(x[:, :40].contiguous())
    assert e.value.status == B.MOE_ERR_UNSUPPORTED and "moe_quantize_int8" in str(e.value)
    with pytest.raises(B.MoeError):
        B.moe_route_backward(x, torch.zeros(4, 9, dtype=torch.int32, device="cuda"),
                             torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError, match="rows must have x's dtype"):
        B.moe_dispatch(x, g, 2, rows=torch.zeros(8, 64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        B.moe_dispatch(x, g, 2, rows=torch.zeros(7, 64, device="cuda"))
    with pytest.raises(ValueError, match="base must have"):
        B.moe_combine(torch.zeros(8, 64, device="cuda"), torch.zeros(4, 2, device="cuda"), g,
                      base=x, y=torch.zeros(4, 64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="expected cuda"):
        B.moe_combine(torch.zeros(8, 64, device="cuda"), torch.zeros(4, 2, device="cuda"), g,
                      base=x.cpu())
    q, s = B.moe_quantize_int8(x)
    w = B.Int8Weight(*on_gpu(int8_weight(1, 8, 32, 64)))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        B.moe_product_int8(w, q, s, g, top_k=2, out_dtype=torch.float16)
    with pytest.raises(B.MoeError):
        B.moe_product_int8(w, q, s)  # several matrices, no grouping
    with pytest.raises(B.MoeError):
        B.moe_swiglu_int8(w, B.Int8Weight(*on_gpu(int8_weight(1, 8, 48, 64))), q, s, g, top_k=2)
    torch.cuda.synchronize()
