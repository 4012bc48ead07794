"""Refusals of the calls on rows in expert order, of the router's gradient and
of the int8 products: every call here fails its checks (or has nothing to do)
before anything reaches a GPU."""

import ctypes

import pytest
import torch

from block_quantized_expert_amd import binding as B

P = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
BIG = 1 << 33
BF16, F32 = B.MOE_ACT_BF16, B.MOE_ACT_F32
OK, INV, UNS = B.MOE_OK, B.MOE_ERR_INVALID, B.MOE_ERR_UNSUPPORTED


def _call(name, order, defaults, changes):
    args = dict(defaults, **changes)
    return getattr(B.lib(), name)(*[args[k] for k in order], None)


DISPATCH = ["x", "type", "xs", "n", "k", "h", "e", "off", "inv", "rows", "rs"]
ROWS_DEFAULTS = dict(x=P, dy=P, rows=P, y=P, base=None, drows=P, dw=P, w=P, type=BF16, ytype=BF16,
                     xs=64, rs=64, bs=64, ys=64, ds=64, n=4, k=2, h=64, e=8, off=P, inv=P)
BACK = ["x", "type", "xs", "n", "k", "h", "inv", "y", "ys"]
COMBINE = ["rows", "type", "rs", "n", "k", "h", "w", "inv", "base", "bs", "y", "ytype", "ys"]
COMBINE_BACK = ["dy", "ytype", "ys", "rows", "type", "rs", "n", "k", "h", "e", "w", "off", "inv",
                "drows", "ds", "dw"]

SIZES = [({"n": -1}, INV), ({"k": 0}, INV), ({"h": 0}, INV), ({"k": 9}, UNS),
         ({"n": (1 << 22) + 1}, UNS), ({"type": 2}, UNS), ({"inv": None}, INV)]


@pytest.mark.parametrize("name,order,changes,expected", [
    (n, o, c, s) for n, o in (("moe_dispatch", DISPATCH), ("moe_dispatch_backward", BACK),
                              ("moe_combine", COMBINE), ("moe_combine_backward", COMBINE_BACK))
    for c, s in SIZES] + [
    ("moe_dispatch", DISPATCH, {"x": None}, INV),
    ("moe_dispatch", DISPATCH, {"x": ODD}, INV),
    ("moe_dispatch", DISPATCH, {"rows": None}, INV),
    ("moe_dispatch", DISPATCH, {"off": None}, INV),
    ("moe_dispatch", DISPATCH, {"e": 0}, INV),
    ("moe_dispatch", DISPATCH, {"e": 1025}, UNS),
    ("moe_dispatch", DISPATCH, {"xs": 63}, INV),
    ("moe_dispatch", DISPATCH, {"rs": 63}, INV),
    ("moe_dispatch", DISPATCH, {"rs": BIG}, UNS),
    ("moe_dispatch", DISPATCH, {"h": 65537, "xs": 65537, "rs": 65537}, UNS),
    ("moe_dispatch_backward", BACK, {"y": None}, INV),
    ("moe_dispatch_backward", BACK, {"ys": 63}, INV),
    ("moe_combine", COMBINE, {"w": None}, INV),
    ("moe_combine", COMBINE, {"ytype": 5}, UNS),
    ("moe_combine", COMBINE, {"ytype": F32, "y": ODD}, INV),
    ("moe_combine", COMBINE, {"base": ODD}, INV),
    ("moe_combine", COMBINE, {"base": P, "bs": 1}, INV),
    ("moe_combine", COMBINE, {"ys": 0}, INV),
    ("moe_combine_backward", COMBINE_BACK, {"dy": None}, INV),
    ("moe_combine_backward", COMBINE_BACK, {"dw": None}, INV),
    ("moe_combine_backward", COMBINE_BACK, {"w": None}, INV),
    ("moe_combine_backward", COMBINE_BACK, {"off": None}, INV),
    ("moe_combine_backward", COMBINE_BACK, {"ytype": -1}, UNS),
    ("moe_combine_backward", COMBINE_BACK, {"ys": 8}, INV),
])
def test_rows_refuse(name, order, changes, expected):
    assert _call(name, order, ROWS_DEFAULTS, changes) == expected


@pytest.mark.parametrize("name,order", [
    ("moe_dispatch", DISPATCH), ("moe_dispatch_backward", BACK), ("moe_combine", COMBINE),
    ("moe_combine_backward", COMBINE_BACK)])
def test_rows_no_tokens_is_a_no_op(name, order):
    nulls = {k: None for k in ("x", "rows", "y", "dy", "drows", "dw", "w", "off", "inv")}
    assert _call(name, order, ROWS_DEFAULTS, dict(nulls, n=0)) == OK


ROUTE = ["l", "ids", "dw", "n", "e", "k", "scale", "dl", "err"]
ROUTE_DEFAULTS = dict(l=P, ids=P, dw=P, n=4, e=16, k=2, scale=1.5, dl=P, err=None)


@pytest.mark.parametrize("changes,expected", [
    ({"l": None}, INV), ({"ids": None}, INV), ({"dw": None}, INV), ({"dl": None}, INV),
    ({"n": -1}, INV), ({"e": 0}, INV), ({"k": 0}, INV), ({"k": 17}, INV), ({"k": 9}, UNS),
    ({"e": 1025}, UNS), ({"scale": 0.0}, INV), ({"scale": float("nan")}, INV),
    ({"scale": float("inf")}, INV), ({"n": 0, "l": None, "dl": None}, OK)])
def test_route_backward_refuses(changes, expected):
    assert _call("moe_route_backward", ROUTE, ROUTE_DEFAULTS, changes) == expected


QUANT = ["x", "type", "xs", "n", "c", "q", "s"]
QUANT_DEFAULTS = dict(x=P, type=BF16, xs=64, n=4, c=64, q=P, s=P)


@pytest.mark.parametrize("changes,expected", [
    ({"x": None}, INV), ({"q": None}, INV), ({"s": None}, INV), ({"q": ODD}, INV),
    ({"x": ODD}, INV), ({"type": 3}, UNS), ({"n": -1}, INV), ({"c": 0}, INV),
    ({"c": 40}, UNS), ({"c": 65552, "xs": 65552}, UNS), ({"xs": 48}, INV),
    ({"n": 0, "x": None, "q": None, "s": None}, OK)])
def test_quantize_refuses(changes, expected):
    assert _call("moe_quantize_int8", QUANT, QUANT_DEFAULTS, changes) == expected


def _weight(e=8, rows=32, cols=64, q=0x10000, scale=0x10000):
    return B.MoeInt8Weight(e, rows, cols, q, scale)


PRODUCT = ["q", "s", "n", "off", "perm", "k", "out", "type", "os"]
PRODUCT_DEFAULTS = dict(q=P, s=P, n=8, off=P, perm=P, k=2, out=P, type=BF16, os=32)


def _product(w, up, changes):
    args = dict(PRODUCT_DEFAULTS, **changes)
    refs = [ctypes.byref(w) if w is not None else None]
    name = "moe_product_int8"
    if up is not False:
        refs.append(ctypes.byref(up) if up is not None else None)
        name = "moe_swiglu_int8"
    return getattr(B.lib(), name)(*refs, *[args[k] for k in PRODUCT], None)


@pytest.mark.parametrize("changes,expected", [
    ({"q": None}, INV), ({"q": ODD}, INV), ({"s": None}, INV), ({"out": None}, INV),
    ({"out": ODD}, INV), ({"n": -1}, INV), ({"k": -1}, INV), ({"k": 9}, UNS),
    ({"n": 9}, INV), ({"perm": None}, INV), ({"type": 2}, UNS), ({"os": 31}, INV),
    ({"off": None}, INV), ({"n": 0, "q": None, "s": None, "out": None, "perm": None}, OK)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_refuses(changes, expected, swiglu):
    assert _product(_weight(), _weight() if swiglu else False, changes) == expected


@pytest.mark.parametrize("weight,expected", [
    ({"e": 0}, INV), ({"rows": 0}, INV), ({"cols": 0}, INV), ({"e": 1025}, UNS),
    ({"cols": 72}, UNS), ({"cols": 65552}, UNS), ({"rows": 65537}, UNS), ({"q": 0}, INV),
    ({"q": 0x10008}, INV), ({"scale": 0}, INV), ({"scale": 0x10002}, INV)])
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
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = tuple(torch.zeros(m, dtype=torch.int32) for m in (8, 9, 8, 8))
    with pytest.raises(ValueError, match="GPU"):
        B.moe_dispatch(x, g, 2)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        B.moe_dispatch(x.half(), g, 2)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        B.moe_dispatch(torch.zeros(64, 4, dtype=torch.bfloat16).t(), g, 2)
    with pytest.raises(ValueError, match="perm"):
        B.moe_dispatch(x, g[:2] + (g[2][:7], g[3]), 2)
    with pytest.raises(ValueError, match="w must be"):
        B.moe_combine(torch.zeros(8, 64), torch.zeros(4, 2).double(), g)
    with pytest.raises(ValueError, match=r"n\*top_k"):
        B.moe_combine(torch.zeros(8, 64), torch.zeros(3, 2), g)
    with pytest.raises(ValueError, match="ids must be"):
        B.moe_route_backward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64),
                             torch.zeros(4, 2))
    with pytest.raises(ValueError, match="int8"):
        B.Int8Weight(torch.zeros(4, 64), torch.zeros(4))
    w = B.Int8Weight(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="64"):
        B.moe_product_int8(w, torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2))
    with pytest.raises(ValueError, match="experts"):
        B.moe_product_int8(w, torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8), g)


def test_binding_refuses_what_is_no_tensor_or_grouping():
    x = torch.zeros(4, 64)
    g = tuple(torch.zeros(m, dtype=torch.int32) for m in (8, 9, 8, 8))
    with pytest.raises(TypeError, match="x must be a tensor"):
        B.moe_dispatch([1.0], g, 2)
    with pytest.raises(ValueError, match="grouping"):
        B.moe_dispatch(x, g[:3], 2)
    with pytest.raises(ValueError, match="grouping"):
        B.moe_dispatch(x, None, 2)
    with pytest.raises(TypeError, match="offsets must be a tensor"):
        B.moe_dispatch(x, (g[0], None, g[2], g[3]), 2)
    with pytest.raises(TypeError):
        B.moe_dispatch(x, g, "2")
    with pytest.raises(ValueError, match="out of range"):
        B.moe_dispatch(x, g, 1 << 40)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        B.moe_quantize_int8(x.double())
    with pytest.raises(ValueError, match="scale must be"):
        B.Int8Weight(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(5))


# Arrays of 4-byte elements that are not where such elements can lie.
@pytest.mark.parametrize("name,order,array", [
    ("moe_dispatch", DISPATCH, "off"), ("moe_dispatch", DISPATCH, "inv"),
    ("moe_dispatch_backward", BACK, "inv"), ("moe_combine", COMBINE, "w"),
    ("moe_combine", COMBINE, "inv"), ("moe_combine_backward", COMBINE_BACK, "w"),
    ("moe_combine_backward", COMBINE_BACK, "off"), ("moe_combine_backward", COMBINE_BACK, "inv"),
    ("moe_combine_backward", COMBINE_BACK, "dw")])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_rows_refuse_misaligned_arrays(name, order, array, at):
    misplaced = ctypes.c_void_p(P.value + at)
    assert _call(name, order, ROWS_DEFAULTS, {array: misplaced}) == INV
    assert _call(name, order, ROWS_DEFAULTS, {array: misplaced, "n": 0}) == OK


@pytest.mark.parametrize("array", ["l", "ids", "dw", "dl", "err"])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_route_backward_refuses_misaligned_arrays(array, at):
    misplaced = ctypes.c_void_p(P.value + at)
    assert _call("moe_route_backward", ROUTE, ROUTE_DEFAULTS, {array: misplaced}) == INV
    assert _call("moe_route_backward", ROUTE, ROUTE_DEFAULTS, {array: misplaced, "n": 0}) == OK


@pytest.mark.parametrize("array", ["off", "perm", "s"])
@pytest.mark.parametrize("at", [1, 2, 3])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_refuses_misaligned_arrays(array, at, swiglu):
    up = _weight() if swiglu else False
    misplaced = ctypes.c_void_p(P.value + at)
    assert _product(_weight(), up, {array: misplaced}) == INV
    assert _product(_weight(), up, {array: misplaced, "n": 0}) == OK


def test_binding_refuses_a_stream_of_another_device():
    # streams stood in for: the check comes before anything is done with one
    class Other:
        device = torch.device("cuda", 1)

    x = torch.zeros(4, 64)
    g = tuple(torch.zeros(m, dtype=torch.int32) for m in (8, 9, 8, 8))
    w = B.Int8Weight(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    q, s = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    for call in (lambda st: B.moe_dispatch(x, g, 2, stream=st),
                 lambda st: B.moe_route_backward(x, g[0], x, stream=st),
                 lambda st: B.moe_quantize_int8(x, stream=st),
                 lambda st: B.moe_product_int8(w, q, s, stream=st),
                 lambda st: B.moe_swiglu_int8(w, w, q, s, stream=st)):
        with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cpu"):
            call(Other())


TILE_SHAPES = [(256, 256), (128, 256), (64, 256), (16, 256), (128, 128), (64, 64)]


@pytest.mark.parametrize("sizes,expected", [
    ((0, 8, 16, 1, 1, 0), INV), ((1, 0, 16, 1, 1, 0), INV), ((1, 8, 0, 1, 1, 0), INV),
    ((1, 8, 16, 0, 1, 0), INV), ((2, 8, 16, 1, 0, 0), INV), ((1025, 8, 16, 1, 1, 0), UNS),
    ((1, 65537, 16, 1, 1, 0), UNS), ((1, 8, 24, 1, 1, 0), UNS), ((1, 8, 65552, 1, 1, 0), UNS),
    ((1, 8, 16, (1 << 25) + 1, 1, 0), UNS)])
def test_int8_form_refuses(sizes, expected):
    out = [ctypes.c_int32() for _ in range(3)]
    assert B.lib().moe_int8_form(*sizes, *[ctypes.byref(v) for v in out]) == expected


def test_int8_form_refuses_null():
    v = ctypes.byref(ctypes.c_int32())
    for null in range(3):
        out = [None if i == null else v for i in range(3)]
        assert B.lib().moe_int8_form(1, 8, 16, 1, 1, 0, *out) == INV


def test_int8_forms_of_few_rows_have_no_persistent_workgroups():
    assert B.moe_int8_form(1, 4096, 4096, 1, False, False) == (16, 16, 0)
    assert B.moe_int8_form(256, 2048, 4096, 6, True, True) == (16, 16, 0)


def test_gpu_cases_take_every_int8_tile_shape_across_tiles():
    """Every tile shape, plain and with SwiGLU, dense and grouped, is chosen by a
    case of test_gpu_int8.py that gives every persistent workgroup two tiles
    and more; where the shape is chosen for reductions of one step, one of those
    has such a reduction."""
    import test_gpu_int8 as G

    reached, one_step = set(), set()

    def look(kind, e, rows, cols, counts, slots):
        for swiglu in (False, True):
            r, c, workgroups = B.moe_int8_form(e, rows, cols, slots, kind == "grouped", swiglu)
            items = sum(-(-int(n) // r) for n in counts) * -(-rows // c)
            if workgroups and items >= 2 * workgroups:
                key = (kind, swiglu, r, c * 2 if swiglu else c)
                reached.add(key)
                if cols <= 128:
                    one_step.add(key[1:])

    for n, rows, cols, _ in G.SEVERAL_TILES:
        look("dense", 1, rows, cols, [n], n)
    for slots, e, share, rows, cols in G.GROUPED_SEVERAL_TILES:
        off = G.several_tiles_offsets(slots, e, share, seed=slots + e)
        look("grouped", e, rows, cols, off[1:] - off[:-1], slots)
    want = {(kind, swiglu, r, c) for kind in ("dense", "grouped") for swiglu in (False, True)
            for r, c in TILE_SHAPES}
    assert reached == want, sorted(want - reached)
    # 256 x 256 tiles are taken for long reductions, 128 x 256 for three steps
    # and more, 128 x 128 of SwiGLU mostly for several
    short = {(swiglu, r, c) for swiglu in (False, True) for r, c in TILE_SHAPES[2:]}
    assert one_step >= short - {(True, 128, 128)}, sorted(short - one_step)
