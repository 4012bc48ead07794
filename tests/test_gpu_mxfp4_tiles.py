"""MXFP4 products at sizes that take every tile shape, with 64-bit references on
the GPU.  Sizes are odd where they can be; reductions are of one step of 256
inputs, of two, the second a part, and of more.  Bounds as in
test_gpu_mxfp4.py."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from rows_testlib import U32, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# rows of the left operand, weight rows, cols
DENSE = [
    (17, 100, 32), (16, 104, 320), (16, 100, 576), (17, 6064, 288), (17, 7029, 224),
    (17, 4067, 704), (65, 8502, 64), (5710, 101, 288), (68, 7234, 544), (34, 8331, 64),
    (269, 6591, 32), (971, 4129, 32), (204, 8503, 288), (577, 6531, 288), (204, 8527, 544),
    (98, 8535, 32), (5953, 648, 544), (67, 8223, 352), (68, 8577, 544), (7225, 2205, 32),
    (513, 6837, 288), (6742, 259, 32), (396, 8953, 544), (1936, 8193, 288), (901, 8871, 800),
    (3897, 4083, 672), (1946, 3985, 64), (7976, 3997, 32), (6559, 4867, 288), (2850, 3524, 288),
    (4017, 3999, 32), (2865, 7042, 288), (2570, 6301, 832), (5038, 6623, 544),
    (306, 193, 288), (17, 2120, 32), (37, 2074, 576), (408, 8280, 64), (5696, 324, 544),
    (6758, 1155, 32), (1836, 4376, 544),
]
# experts, slots, weight rows, cols
GROUPED = [
    (1, 17, 103, 32), (1, 17, 109, 352), (1, 18, 100, 544), (150, 122, 244, 32),
    (64, 2045, 165, 32), (1, 1996, 119, 384), (1, 1222, 164, 576), (40, 51, 742, 288),
    (256, 547, 102, 608), (150, 205, 215, 32), (256, 3652, 130, 352), (64, 2002, 702, 32),
    (256, 2820, 148, 576), (1, 7381, 540, 32), (3, 2239, 137, 256), (150, 7520, 199, 288),
    (1, 5243, 779, 288), (40, 2609, 1345, 32), (40, 7387, 522, 544), (256, 5970, 600, 32),
    (40, 1249, 1209, 544), (64, 5536, 324, 608), (64, 3718, 811, 288), (256, 7488, 562, 96),
    (256, 7525, 548, 288), (150, 2807, 1290, 288), (5, 5131, 1540, 32), (1, 4690, 3597, 32),
    (256, 7788, 263, 96), (5, 7435, 2226, 288), (150, 5144, 817, 640), (40, 7597, 1045, 320),
    (256, 5889, 656, 608), (150, 7364, 283, 384), (3, 4013, 2108, 544), (150, 7473, 279, 608),
    (40, 1964, 4613, 576), (256, 6960, 1063, 32), (1, 7054, 4613, 576), (5, 4632, 7185, 32),
    (150, 6954, 1032, 320), (1, 5890, 5643, 288), (5, 4744, 3548, 544), (1024, 7900, 300, 544),
    (1024, 2001, 211, 160), (3, 54, 1290, 32), (5, 546, 123, 288), (1, 608, 128, 544),
    (64, 2897, 3107, 288), (256, 5805, 209, 544), (40, 3094, 656, 544), (150, 6739, 1161, 32),
    (150, 6641, 1066, 544), (40, 3515, 4843, 32), (1, 7469, 1048, 800), (40, 3608, 4700, 288),
    (64, 5763, 2888, 608), (1, 611, 115, 320), (1, 764, 102, 576),
]


def counts_of(e, slots):
    """Rows of each expert: uneven, a tenth of the experts without any; one slot
    in twenty has no expert."""
    rng = np.random.default_rng(e + slots)
    share = rng.random(e) + 0.2
    share[rng.random(e) < 0.1] = 0
    share[rng.integers(e)] = 1
    return rng.multinomial(slots - slots // 20, share / share.sum())


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


def _random(seed, *shape, mid=127, spread=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    *lead, c = shape
    codes = torch.randint(0, 256, (*lead, c // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(mid - spread, mid + spread + 1, (*lead, c // 32), generator=g,
                           device="cuda", dtype=torch.uint8)
    return codes, scales


def _values(codes, scales):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    lut = torch.cat([lut, -lut])
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def _words(scales):
    n, b = scales.shape
    words = -(-b // 16)
    out = torch.zeros(n, words * 16, dtype=torch.uint8, device="cuda")
    out[:, :b] = scales
    return out.view(n, words, 16).transpose(0, 1).contiguous()


def _out(n, rows, dtype, aligned):
    """(rows to write into, their gaps): strides of whole 16 bytes or not."""
    stride = rows + (-rows % 8 if aligned else 3)
    buf = torch.full((n * stride + 1,), 7.0, dtype=dtype, device="cuda")
    buf = buf[:-1] if aligned else buf[1:]
    buf = buf.view(n, stride)
    return buf[:, :rows], buf[:, rows:]


def _product(w, x, offsets, left):
    """(out, its error before the last rounding) in fp64."""
    out = torch.zeros(len(left), w[0].shape[1], dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    cols = w[0].shape[2] * 2
    for e in range(w[0].shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b <= a:
            continue
        v, wv = _values(x[0][left[a:b]], x[1][left[a:b]]), _values(w[0][e], w[1][e])
        out[a:b] = v @ wv.t().contiguous()
        sums = v.abs() @ wv.abs().t().contiguous()
        unit = torch.exp2(x[1][left[a:b]].amin(1).double() - 127)[:, None] * torch.exp2(
            w[1][e].amin(1).double() - 127) / 4
        err[a:b] = torch.where(sums < 2.0 ** 24 * unit, 0.0, (cols / 32 + 8) * 2.0 ** -20 * sums)
    return out, err


def _within(got, ref, err, what):
    # below the normal numbers a step is a fixed one: half of bf16's 2^-133, of fp32's 2^-149
    bound = err + half_step(got.dtype) * (ref.abs() + err)
    bound = bound + (2.0 ** -134 if got.dtype == BF16 else 0) + 2.0 ** -149
    over = (got.double() - ref).abs() - bound
    assert bool(torch.isfinite(got).all()) and float(over.max()) <= 0, what


def _within_swiglu(got, g, gerr, u, uerr, what):
    sig = torch.exp(-torch.logaddexp(torch.zeros_like(g), -g))
    y = g * sig * u
    err = (2 * g.abs() + 10) * U32 * y.abs()
    err = err + 1.1 * gerr * u.abs() + uerr * (g * sig).abs() + 2 * gerr * uerr
    _within(got, y, err + torch.where(g < -86.9, 1.5e-36 * u.abs(), 0.0), what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,cols", DENSE)
def test_dense_products_of_every_tile_shape(n, rows, cols, dtype):
    print("case dense", n, rows, cols, dtype, flush=True)
    w, u, x = _random(1, 1, rows, cols, mid=124), _random(2, 1, rows, cols, mid=124), _random(
        3, n, cols)
    gw, gu = B.Mxfp4Weight(*w), B.Mxfp4Weight(*u)
    left = x[0], _words(x[1])
    every = torch.arange(n, device="cuda")
    a, b = _product(w, x, [0, n], every), _product(u, x, [0, n], every)
    out, gap = _out(n, rows, dtype, dtype == BF16)
    B.moe_product_mxfp4(gw, *left, out=out)
    _within(out, *a, "product")
    assert bool((gap == 7).all())
    out, gap = _out(n, rows, dtype, dtype == F32)
    B.moe_swiglu_mxfp4(gw, gu, *left, out=out)
    _within_swiglu(out, *a, *b, "swiglu")
    assert bool((gap == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("e,slots,rows,cols", GROUPED)
def test_grouped_products_of_every_tile_shape(e, slots, rows, cols, dtype):
    print("case grouped", e, slots, rows, cols, dtype, flush=True)
    k = 3 if slots % 3 == 0 else 2 if slots % 2 == 0 else 1
    counts = counts_of(e, slots)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = int(offsets[-1])
    perm = np.random.default_rng(slots).permutation(slots).astype(np.int32)
    g = tuple(torch.from_numpy(v).cuda() for v in (counts.astype(np.int32), offsets, perm, perm))
    w, u = _random(1, e, rows, cols, mid=124), _random(2, e, rows, cols, mid=124)
    gw, gu = B.Mxfp4Weight(*w), B.Mxfp4Weight(*u)
    # tokens that the slots gather, SwiGLU
    x = _random(3, slots // k, cols)
    left = torch.div(g[2].long(), k, rounding_mode="floor")
    a, b = _product(w, x, offsets, left), _product(u, x, offsets, left)
    out, gap = _out(slots, rows, dtype, dtype == F32)
    B.moe_swiglu_mxfp4(gw, gu, x[0], _words(x[1]), g, top_k=k, out=out)
    _within_swiglu(out, *a, *b, "swiglu")
    assert bool((gap == 7).all()) and not bool(out[total:].any())
    # rows in expert order, those behind the last expert's not finite
    x = _random(4, slots, cols)
    ref = _product(u, x, offsets, torch.arange(slots, device="cuda"))
    x[1][total:] = 255
    out, gap = _out(slots, rows, dtype, dtype == BF16)
    B.moe_product_mxfp4(gu, x[0], _words(x[1]), g, out=out)
    _within(out, *ref, "product")
    assert bool((gap == 7).all()) and not bool(out[total:].any())


def test_gathered_rows_past_four_gigabytes():
    # 140000 tokens of 32768 bytes of codes; only some hold anything
    n, c = 140000, 65536
    codes = torch.zeros(n, c // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((c // 512, n, 16), 127, dtype=torch.uint8, device="cuda")
    look = torch.tensor([0, 1, 65535, 131071, 131072, 131073, n - 1], device="cuda")
    some = _random(5, len(look), c)
    codes[look], scales[:, look] = some[0], _words(some[1])
    w = _random(6, 2, 24, c, mid=124)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(1)).int().cuda()
    inverse = torch.empty_like(perm)
    inverse[perm.long()] = torch.arange(n, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 70001, n], dtype=torch.int32, device="cuda")
    grouping = (offsets.diff().int(), offsets, perm, inverse)
    out = B.moe_product_mxfp4(B.Mxfp4Weight(*w), codes, scales, grouping, top_k=1, out_dtype=F32)
    at = inverse[look].long()
    for i in range(len(look)):
        e = int(at[i] >= 70001)
        one = (w[0][e:e + 1], w[1][e:e + 1])
        ref = _product(one, (some[0][i:i + 1], some[1][i:i + 1]), [0, 1], torch.tensor([0]))
        _within(out[at[i]:at[i] + 1], *ref, i)
    out[at] = 0
    assert not bool(out.any())
    del codes, scales, out
    torch.cuda.empty_cache()


def test_tiled_products_in_a_graph_follow_their_inputs():
    # one capture; the rows, the counts and the gather change between replays
    n, k, e, rows, cols = 1100, 3, 24, 530, 1056
    slots = n * k
    gate, up = (B.Mxfp4Weight(*_random(i, e, rows, cols, mid=124)) for i in (1, 2))
    down = B.Mxfp4Weight(*_random(3, e, 200, 32 * (rows // 32), mid=124))
    assert B.moe_mxfp4_form(e, rows, cols, slots, True, True)[2] > 0
    x = torch.randn(n, cols, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    perm = torch.arange(slots, dtype=torch.int32, device="cuda")
    g = (offsets[:e], offsets, perm, perm)

    def deal(seed):
        counts = np.random.default_rng(seed).multinomial(slots - 100 * seed, np.ones(e) / e)
        counts[seed] = 0
        offsets.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).int())
        perm.copy_(torch.randperm(slots, generator=torch.Generator().manual_seed(seed)).int())
        x.copy_(torch.roll(x, 1, 0) * 1.25)

    def passes():
        h = B.moe_swiglu_mxfp4(gate, up, *B.moe_quantize_mxfp4(x), g, top_k=k)
        h = h[:, :32 * (rows // 32)]
        return h, B.moe_product_mxfp4(down, *B.moe_quantize_mxfp4(h), g, out_dtype=F32)

    deal(1)
    passes()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = passes()
    for seed in range(4):
        deal(seed)
        want = [t.clone() for t in passes()]
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed
        total = int(offsets[-1])
        assert bool(want[1][:total].any()) and not bool(want[1][total:].any())
