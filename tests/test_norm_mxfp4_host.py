"""Refusals of the RMS norm's calls and of the MXFP4 rows and products: every
call here fails its checks (or has nothing to do) before anything reaches a
GPU.  The 64-bit references of both are held against the formats' definition."""

import ctypes

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from mxfp4_testlib import E2M1, SIGNED, norm_back_ref, norm_ref, quantize_ref, values

P = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)
BIG = 1 << 33
BF16, F32 = B.MOE_ACT_BF16, B.MOE_ACT_F32
OK, INV, UNS, WSP = B.MOE_OK, B.MOE_ERR_INVALID, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
EPS = 1e-6


def _rows(**changes):
    r = dict(n_rows=4, hidden=64, eps=EPS, x=0x10000, x_type=BF16, x_stride=64, weight=0x10000,
             w_type=F32, residual=0x10000, res_type=BF16, res_stride=64, total=0x10000,
             total_stride=64)
    r.update(changes)
    return B.MoeNormRows(**r)


ROWS = [({"n_rows": -1}, INV), ({"hidden": 0}, INV), ({"eps": 0.0}, INV), ({"eps": -1.0}, INV),
        ({"eps": float("nan")}, INV), ({"eps": float("inf")}, INV),
        ({"n_rows": (1 << 25) + 1}, UNS), ({"x_type": 2}, UNS), ({"w_type": 2}, UNS),
        ({"res_type": -1}, UNS), ({"x": 0}, INV), ({"x": 0x10001}, INV), ({"weight": 0}, INV),
        ({"weight": 0x10002}, INV), ({"residual": 0x10001}, INV), ({"total": 0}, INV),
        ({"total": 0x10001}, INV), ({"x_stride": 63}, INV), ({"x_stride": BIG}, UNS),
        ({"res_stride": 63}, INV), ({"total_stride": 63}, INV), ({"total_stride": BIG}, UNS),
        ({"hidden": 65568, "x_stride": 65568, "res_stride": 65568, "total_stride": 65568}, UNS)]


@pytest.mark.parametrize("changes,expected", ROWS)
def test_norm_refuses_rows(changes, expected):
    L, r = B.lib(), ctypes.byref(_rows(**changes))
    assert L.moe_rmsnorm(r, P, BF16, 70000, None) == expected
    assert L.moe_rmsnorm_int8(r, P, P, None) == expected
    assert L.moe_rmsnorm_mxfp4(r, P, P, None) == expected


def test_norm_refuses_outputs():
    L, r = B.lib(), ctypes.byref(_rows())
    assert L.moe_rmsnorm(None, P, BF16, 64, None) == INV
    assert L.moe_rmsnorm_int8(None, P, P, None) == INV
    assert L.moe_rmsnorm_mxfp4(None, P, P, None) == INV
    assert L.moe_rmsnorm(r, None, BF16, 64, None) == INV
    assert L.moe_rmsnorm(r, ODD, BF16, 64, None) == INV
    assert L.moe_rmsnorm(r, ctypes.c_void_p(0x10002), F32, 64, None) == INV
    assert L.moe_rmsnorm(r, P, 2, 64, None) == UNS
    assert L.moe_rmsnorm(r, P, BF16, 63, None) == INV
    assert L.moe_rmsnorm(r, P, BF16, BIG, None) == UNS
    for f in (L.moe_rmsnorm_int8, L.moe_rmsnorm_mxfp4):
        for bad in (None, HALF):
            assert f(r, bad, P, None) == INV
    assert L.moe_rmsnorm_int8(r, P, None, None) == INV
    assert L.moe_rmsnorm_int8(r, P, ctypes.c_void_p(0x10002), None) == INV
    assert L.moe_rmsnorm_mxfp4(r, P, HALF, None) == INV
    assert L.moe_rmsnorm_int8(ctypes.byref(_rows(hidden=56)), P, P, None) == UNS
    assert L.moe_rmsnorm_mxfp4(ctypes.byref(_rows(hidden=48)), P, P, None) == UNS


def test_norm_without_rows_is_a_no_op():
    L = B.lib()
    r = ctypes.byref(_rows(n_rows=0, x=0, weight=0, residual=0, total=0))
    assert L.moe_rmsnorm(r, None, BF16, 64, None) == OK
    assert L.moe_rmsnorm_int8(r, None, None, None) == OK
    assert L.moe_rmsnorm_mxfp4(r, None, None, None) == OK


BACK = ["dy", "dyt", "dys", "s", "st", "ss", "w", "wt", "t", "ts", "n", "h", "eps", "dx", "dxs",
        "dw", "ws", "bytes"]
BACK_DEFAULTS = dict(dy=P, dyt=BF16, dys=64, s=P, st=BF16, ss=64, w=P, wt=F32, t=P, ts=64, n=4,
                     h=64, eps=EPS, dx=P, dxs=64, dw=P, ws=P, bytes=1 << 20)


@pytest.mark.parametrize("changes,expected", [
    ({"dy": None}, INV), ({"dy": ODD}, INV), ({"s": None}, INV), ({"s": ODD}, INV),
    ({"w": None}, INV), ({"t": ODD}, INV), ({"dx": None}, INV), ({"dx": ODD}, INV),
    ({"dyt": 2}, UNS), ({"st": 2}, UNS), ({"wt": 2}, UNS), ({"n": -1}, INV), ({"h": 0}, INV),
    ({"h": 65537, "dys": 65537, "ss": 65537, "ts": 65537, "dxs": 65537}, UNS),
    ({"n": (1 << 25) + 1}, UNS), ({"eps": 0.0}, INV), ({"eps": float("nan")}, INV),
    ({"dys": 63}, INV), ({"ss": 63}, INV), ({"ts": 63}, INV), ({"dxs": 63}, INV),
    ({"dys": BIG}, UNS), ({"dxs": BIG}, UNS), ({"dw": ODD}, INV), ({"ws": None}, WSP),
    ({"bytes": 255}, WSP), ({"ws": ctypes.c_void_p(0x10004)}, INV),
    ({"n": 0, "dy": None, "s": None, "w": None, "t": None, "dx": None, "dw": None, "ws": None}, OK)])
def test_norm_backward_refuses(changes, expected):
    args = dict(BACK_DEFAULTS, **changes)
    assert B.lib().moe_rmsnorm_backward(*[args[k] for k in BACK], None) == expected


def test_norm_backward_workspace():
    f = B.lib().moe_rmsnorm_backward_workspace_bytes
    assert f(0, 64) == f(-1, 64) == f(4, 0) == 0
    assert f(1, 64) == 4 * 64
    assert f(1 << 25, 4096) < 1 << 25
    # rows longer than the registers hold keep r
    assert f(1000, 8192) < f(1000, 8193) + 8192 * 4 * 256
    assert f(1001, 16384) >= 1001 * 4 + 16384 * 4


QUANT = ["x", "type", "xs", "n", "c", "codes", "scales"]
QUANT_DEFAULTS = dict(x=P, type=BF16, xs=64, n=4, c=64, codes=P, scales=P)


@pytest.mark.parametrize("changes,expected", [
    ({"x": None}, INV), ({"codes": None}, INV), ({"scales": None}, INV), ({"codes": HALF}, INV),
    ({"scales": HALF}, INV), ({"x": ODD}, INV), ({"type": 3}, UNS), ({"n": -1}, INV),
    ({"c": 0}, INV), ({"c": 48}, UNS), ({"c": 65568, "xs": 65568}, UNS), ({"xs": 48}, INV),
    ({"xs": BIG}, UNS), ({"n": (1 << 25) + 1}, UNS),
    ({"n": 0, "x": None, "codes": None, "scales": None}, OK)])
def test_rounding_refuses(changes, expected):
    a = dict(QUANT_DEFAULTS, **changes)
    assert B.lib().moe_quantize_mxfp4(*[a[k] for k in QUANT], None) == expected
    order = ["codes", "scales", "n", "c", "x", "type", "xs"]
    assert B.lib().moe_dequantize_mxfp4(*[a[k] for k in order], None) == expected


def _weight(e=8, rows=32, cols=64, codes=0x10000, scales=0x10000):
    return B.MoeMxfp4Weight(e, rows, cols, codes, scales)


PRODUCT = ["codes", "scales", "n", "off", "perm", "k", "out", "type", "os"]
PRODUCT_DEFAULTS = dict(codes=P, scales=P, n=8, off=P, perm=P, k=2, out=P, type=BF16, os=32)


def _product(w, up, changes):
    args = dict(PRODUCT_DEFAULTS, **changes)
    refs = [ctypes.byref(w) if w is not None else None]
    name = "moe_product_mxfp4"
    if up is not False:
        refs.append(ctypes.byref(up) if up is not None else None)
        name = "moe_swiglu_mxfp4"
    return getattr(B.lib(), name)(*refs, *[args[k] for k in PRODUCT], None)


@pytest.mark.parametrize("changes,expected", [
    ({"codes": None}, INV), ({"codes": HALF}, INV), ({"scales": None}, INV),
    ({"scales": HALF}, INV), ({"out": None}, INV), ({"out": ODD}, INV),
    ({"out": ctypes.c_void_p(0x10002), "type": F32}, INV), ({"n": -1}, INV), ({"k": -1}, INV),
    ({"k": 9}, UNS), ({"n": 9}, INV), ({"perm": None}, INV), ({"type": 2}, UNS),
    ({"os": 31}, INV), ({"os": BIG}, UNS), ({"off": None}, INV),
    ({"off": ctypes.c_void_p(0x10002)}, INV), ({"perm": ctypes.c_void_p(0x10001)}, INV),
    ({"n": (1 << 25) + 2}, UNS),
    ({"n": 0, "codes": None, "scales": None, "out": None, "perm": None}, OK)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_refuses(changes, expected, swiglu):
    assert _product(_weight(), _weight() if swiglu else False, changes) == expected


@pytest.mark.parametrize("weight,expected", [
    ({"e": 0}, INV), ({"rows": 0}, INV), ({"cols": 0}, INV), ({"e": 1025}, UNS),
    ({"cols": 80}, UNS), ({"cols": 65568}, UNS), ({"rows": 65537}, UNS), ({"codes": 0}, INV),
    ({"codes": 0x10008}, INV), ({"scales": 0}, INV), ({"scales": 0x10008}, INV)])
def test_product_refuses_weights(weight, expected):
    assert _product(_weight(**weight), False, {"os": 70000}) == expected
    assert _product(_weight(), _weight(**weight), {"os": 70000}) == expected


def test_product_refuses_pairs_and_null():
    assert _product(None, False, {}) == INV
    assert _product(_weight(), None, {}) == INV
    assert _product(_weight(), _weight(rows=48), {}) == INV
    assert _product(_weight(), _weight(cols=128), {}) == INV
    # dense: one matrix, nothing to gather by
    assert _product(_weight(e=2), False, {"off": None, "k": 0}) == INV
    assert _product(_weight(e=1), False, {"off": None, "k": 2}) == INV


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x, w = torch.zeros(4, 64), torch.ones(64)
    for f in (B.moe_rmsnorm, B.moe_rmsnorm_int8, B.moe_rmsnorm_mxfp4):
        with pytest.raises(ValueError, match="GPU"):
            f(x, w)
        with pytest.raises(ValueError, match="weight must be"):
            f(x, w[:60])
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            f(x.half(), w)
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            f(x, w.double())
        with pytest.raises(ValueError, match="rows must be contiguous"):
            f(torch.zeros(64, 4).t(), w)
        with pytest.raises(TypeError, match="weight must be a tensor"):
            f(x, None)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_rmsnorm_backward(x, x, w)
    with pytest.raises(ValueError, match="shape"):
        B.moe_rmsnorm_backward(x[:3], x, w)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_quantize_mxfp4(x)
    with pytest.raises(ValueError, match="x must be a matrix"):
        B.moe_quantize_mxfp4(w)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_dequantize_mxfp4(codes, scales)
    with pytest.raises(ValueError, match="scales must be"):
        B.moe_dequantize_mxfp4(codes, scales[:, :, :8])
    with pytest.raises(ValueError, match="codes must be"):
        B.moe_dequantize_mxfp4(codes.to(torch.int8), scales)
    with pytest.raises(ValueError, match="codes must be"):
        B.Mxfp4Weight(codes.to(torch.int8), scales)
    with pytest.raises(ValueError, match="scales must be"):
        B.Mxfp4Weight(codes, torch.zeros(4, 1, dtype=torch.uint8))
    weight = B.Mxfp4Weight(codes, torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        B.moe_product_mxfp4(weight, codes, scales)
    with pytest.raises(ValueError, match="codes must be"):
        B.moe_product_mxfp4(weight, codes[:, :16].contiguous(), scales)
    g = tuple(torch.zeros(m, dtype=torch.int32) for m in (8, 9, 4, 4))
    with pytest.raises(ValueError, match="experts"):
        B.moe_product_mxfp4(weight, codes, scales, g)


def test_binding_refuses_a_stream_of_another_device():
    # streams stood in for: the check comes before anything is done with one
    class Other:
        device = torch.device("cuda", 1)

    x, w = torch.zeros(4, 64), torch.ones(64)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, 16, dtype=torch.uint8)
    weight = B.Mxfp4Weight(codes, torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda st: B.moe_rmsnorm(x, w, stream=st),
                 lambda st: B.moe_rmsnorm_int8(x, w, stream=st),
                 lambda st: B.moe_rmsnorm_mxfp4(x, w, stream=st),
                 lambda st: B.moe_rmsnorm_backward(x, x, w, stream=st),
                 lambda st: B.moe_quantize_mxfp4(x, stream=st),
                 lambda st: B.moe_dequantize_mxfp4(codes, scales, stream=st),
                 lambda st: B.moe_product_mxfp4(weight, codes, scales, stream=st),
                 lambda st: B.moe_swiglu_mxfp4(weight, weight, codes, scales, stream=st)):
        with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cpu"):
            call(Other())


def test_weight_lays_scales_out_by_words():
    rows = torch.arange(2 * 3 * 34, dtype=torch.int64).reshape(2, 3, 34).to(torch.uint8)
    w = B.Mxfp4Weight(torch.zeros(2, 3, 544, dtype=torch.uint8), rows)
    assert w.scales.shape == (2, 3, 3, 16)
    for e in range(2):
        for r in range(3):
            got = w.scales[e, :, r].reshape(-1)
            assert torch.equal(got[:34], rows[e, r]) and not got[34:].any()
    assert torch.equal(B.mxfp4_scale_rows(w.scales[1].contiguous(), 1088), rows[1])


def test_reference_rounds_as_the_format_says():
    # by search over the 16 codes: the nearest value, the even code on a tie
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 64)) * np.exp2(rng.integers(-130, 120, (6, 1)).astype(float))
    x[0, :32] = 0
    x[1, :8] = x[1, 8] * np.array([1, 0.5, 0.25, 0.125, 0.625, 0.75, 0.375, -0.875])
    codes, scales = quantize_ref(x)
    got = values(codes, scales)
    for i in range(6):
        for b in range(2):
            v = x[i, 32 * b:32 * b + 32]
            a = np.abs(v).max()
            e = int(np.clip(np.floor(np.log2(a)) - 2, -125, 125)) if a > 0 else -125
            assert scales[i, b] == 127 + e
            for j, t in enumerate(v / 2.0 ** e):
                t = np.clip(t, -6, 6)
                far = np.abs(SIGNED - t)
                best = [c for c in range(16) if far[c] == far.min()]
                if len({abs(SIGNED[c]) for c in best}) > 1:
                    best = [c for c in best if c % 2 == 0]
                assert got[i, 32 * b + j] == SIGNED[best[0]] * 2.0 ** e
    assert E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_reference_gradients_are_the_differences():
    rng = np.random.default_rng(2)
    s, w, dy = rng.standard_normal((2, 5)), rng.standard_normal(5), rng.standard_normal((2, 5))
    dx, dw = norm_back_ref(dy, s, w, EPS)
    d = 2.0 ** -17

    def loss(s, w):
        return (dy * norm_ref(s, w, EPS)[0]).sum()

    for i in range(2):
        for j in range(5):
            t = np.zeros((2, 5))
            t[i, j] = d
            assert abs((loss(s + t, w) - loss(s - t, w)) / (2 * d) - dx[i, j]) < 1e-7
    for j in range(5):
        t = np.zeros(5)
        t[j] = d
        assert abs((loss(s, w + t) - loss(s, w - t)) / (2 * d) - dw[j]) < 1e-7


@pytest.mark.parametrize("sizes,expected", [
    ((0, 8, 32, 1, 1, 0), INV), ((1, 0, 32, 1, 1, 0), INV), ((1, 8, 0, 1, 1, 0), INV),
    ((1, 8, 32, 0, 1, 0), INV), ((2, 8, 32, 1, 0, 0), INV), ((1025, 8, 32, 1, 1, 0), UNS),
    ((1, 65537, 32, 1, 1, 0), UNS), ((1, 8, 48, 1, 1, 0), UNS), ((1, 8, 65568, 1, 1, 0), UNS),
    ((1, 8, 32, (1 << 25) + 1, 1, 0), UNS)])
def test_mxfp4_form_refuses(sizes, expected):
    out = [ctypes.c_int32() for _ in range(3)]
    assert B.lib().moe_mxfp4_form(*sizes, *[ctypes.byref(v) for v in out]) == expected


def test_mxfp4_form_refuses_null():
    v = ctypes.byref(ctypes.c_int32())
    for null in range(3):
        out = [None if i == null else v for i in range(3)]
        assert B.lib().moe_mxfp4_form(1, 8, 32, 1, 1, 0, *out) == INV


def test_gpu_cases_take_every_mxfp4_form():
    """Cases of test_gpu_mxfp4_tiles.py take every form, plain and with SwiGLU,
    dense and grouped, with a reduction of one step and of several; and every
    tile shape with two tiles and more for each persistent workgroup, where it
    is chosen for so many (dense, the small shapes are not)."""
    import test_gpu_mxfp4_tiles as G

    tiles = [(256, 256), (128, 256), (64, 256), (32, 256), (128, 128), (64, 64)]
    few = {False: [(16, 16), (32, 16), (32, 32)], True: [(16, 32), (32, 32)]}
    reached, several = set(), set()

    def look(kind, e, rows, cols, counts, slots):
        for swiglu in (False, True):
            r, c, workgroups = B.moe_mxfp4_form(e, rows, cols, slots, kind == "grouped", swiglu)
            form = (r, c * 2 if swiglu else c)
            reached.add((kind, swiglu, form, cols <= 256))
            items = sum(-(-int(n) // r) for n in counts) * -(-rows // c)
            if workgroups and items >= 2 * workgroups:
                several.add((kind, swiglu, form))

    for n, rows, cols in G.DENSE:
        look("dense", 1, rows, cols, [n], n)
    for e, slots, rows, cols in G.GROUPED:
        look("grouped", e, rows, cols, G.counts_of(e, slots), slots)
    want = {(kind, swiglu, form, one) for kind in ("dense", "grouped") for swiglu in (False, True)
            for form in tiles + few[swiglu] for one in (False, True)}
    assert reached == want, (want - reached, reached - want)
    want = {("grouped", swiglu, form) for swiglu in (False, True) for form in tiles}
    want |= {("dense", swiglu, form) for swiglu in (False, True)
             for form in tiles[:2] + [(128, 128)]}
    assert several >= want, want - several
