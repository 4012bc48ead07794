"""Rows into expert order and back, their gradients and the router's
gradient, against 64-bit references.

Bounds: an output rounds once to its type (half a step); a sum of m fp32
products taken one after the other is off by at most m half-steps of the sum of the
terms' magnitudes (each step rounds a partial sum no larger than that, and the
bounds below count a few steps more than the longest chain has)."""

import numpy as np
import pytest
import torch

from block_quantized_expert_amd import binding as B
from rows_testlib import (U32, assert_within, group, half_step, make_ids, normal, on_gpu,
                          route_backward_ref, strided)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.empty_cache()


# tokens, top_k, experts, hidden, share of dropped slots, row padding
SHAPES = [
    (1, 1, 1, 1, 0.0, 0),
    (1, 6, 256, 4096, 0.0, 0),
    (1, 8, 8, 8, 0.0, 3),
    (3, 2, 5, 7, 0.5, 1),
    (5, 3, 1024, 129, 0.0, 0),
    (33, 4, 16, 2048, 0.3, 8),
    (64, 2, 16, 2059, 0.2, 5),
    (100, 5, 37, 1000, 0.0, 0),
    (257, 7, 64, 515, 0.4, 1),
    (40, 6, 12, 64, 1.0, 0),       # no slot has an expert
    (2, 2, 4, 65536, 0.25, 0),     # the widest row
]


def _case(n, k, e, drop):
    ids = make_ids(n, k, e, drop, seed=n * 31 + k)
    g = group(ids, e)
    return ids, g, on_gpu(g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,h,drop,pad", SHAPES)
def test_dispatch_copies_every_row(n, k, e, h, drop, pad, dtype):
    print("case dispatch", n, k, e, h, drop, pad, dtype, flush=True)
    ids, (_, off, perm, inv), g = _case(n, k, e, drop)
    x = normal(1, n, h, dtype=dtype)
    x.view(-1)[0] = float("inf")  # copied as it is
    rows = strided(torch.zeros(n * k, h, dtype=dtype, device="cuda"), pad).fill_(float("nan"))
    got = B.moe_dispatch(strided(x.cuda(), pad), g, k, rows=rows)
    ref = torch.zeros(n * k, h, dtype=dtype)
    total = int(off[-1])
    ref[:total] = x[torch.from_numpy(perm[:total]).long() // k]
    torch.cuda.synchronize()
    assert got is rows and torch.equal(rows.cpu(), ref)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k,e,h,drop,pad", SHAPES)
def test_dispatch_backward_sums_a_tokens_rows(n, k, e, h, drop, pad, dtype):
    print("case dispatch_backward", n, k, e, h, drop, pad, dtype, flush=True)
    ids, (_, off, perm, inv), g = _case(n, k, e, drop)
    d = normal(2, n * k, h, dtype=dtype)
    d[int(off[-1]):] = float("nan")  # rows that no slot has are not read
    got = B.moe_dispatch_backward(strided(d.cuda(), pad), g, k)
    ref, mag = np.zeros((n, h)), np.zeros((n, h))
    for f in range(n * k):
        if inv[f] >= 0:
            v = d[inv[f]].double().numpy()
            ref[f // k] += v
            mag[f // k] += np.abs(v)
    err = (k + 1) * U32 * mag
    assert_within(got, ref, err + half_step(dtype) * (np.abs(ref) + err), "dx")


@pytest.mark.parametrize("dtype,y_dtype,base", [(BF16, BF16, True), (BF16, F32, False),
                                                (F32, F32, True), (F32, BF16, False)])
@pytest.mark.parametrize("n,k,e,h,drop,pad", SHAPES)
def test_combine_weighs_and_sums(n, k, e, h, drop, pad, dtype, y_dtype, base):
    print("case combine", n, k, e, h, drop, pad, dtype, y_dtype, base, flush=True)
    ids, (_, off, perm, inv), g = _case(n, k, e, drop)
    rows = normal(3, n * k, h, dtype=dtype)
    rows[int(off[-1]):] = float("nan")
    w = normal(4, n, k)
    w.view(-1)[torch.from_numpy(inv < 0)] = float("inf")  # left out whatever it is
    b = normal(5, n, h, dtype=y_dtype) if base else None
    got = B.moe_combine(strided(rows.cuda(), pad), w.cuda(), g,
                        base=strided(b.cuda(), pad) if base else None, y_dtype=y_dtype)
    assert got.dtype == y_dtype
    ref = b.double().numpy().copy() if base else np.zeros((n, h))
    mag = np.abs(ref)
    for f in range(n * k):
        if inv[f] >= 0:
            v = rows[inv[f]].double().numpy() * float(w.view(-1)[f])
            ref[f // k] += v
            mag[f // k] += np.abs(v)
    err = (k + 1) * U32 * mag
    assert_within(got, ref, err + half_step(y_dtype) * (np.abs(ref) + err), "y")


@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("n,k,e,h,drop,pad", SHAPES)
def test_combine_backward(n, k, e, h, drop, pad, dtype, y_dtype):
    print("case combine_backward", n, k, e, h, drop, pad, dtype, y_dtype, flush=True)
    ids, (_, off, perm, inv), g = _case(n, k, e, drop)
    total = int(off[-1])
    rows = normal(6, n * k, h, dtype=dtype)
    rows[total:] = float("nan")
    dy, w = normal(7, n, h, dtype=y_dtype), normal(8, n, k)
    w.view(-1)[torch.from_numpy(inv < 0)] = float("nan")
    drows, dw = B.moe_combine_backward(strided(dy.cuda(), pad), strided(rows.cuda(), pad),
                                       w.cuda(), g)
    d64, r64, w64 = dy.double().numpy(), rows.double().numpy(), w.double().numpy().reshape(-1)
    ref = np.zeros((n * k, h))
    f = perm[:total]
    ref[:total] = w64[f, None] * d64[f // k]
    assert_within(drows, ref, np.abs(ref) * (U32 + half_step(dtype) * (1 + U32)), "drows")
    dots, mag = np.zeros(n * k), np.zeros(n * k)
    for f in range(n * k):
        if inv[f] >= 0:
            terms = d64[f // k] * r64[inv[f]]
            dots[f], mag[f] = terms.sum(), np.abs(terms).sum()
    # the longest chain: a lane's own columns, the lanes of a wavefront (6
    # steps) and the wavefronts (4)
    chain = 8 * -(-h // 1024) + 10
    assert_within(dw, dots.reshape(n, k), (chain * U32 * mag).reshape(n, k), "dw")


def test_gradients_match_differences():
    # y is linear in the rows and in the weights: a difference of two calls is
    # the directional derivative up to rounding.  fp32 sums of 6 terms of order
    # 1 (10 for a row's sum of 64) are off by 2^-20 or so each
    n, k, e, h = 17, 6, 32, 64
    _, _, g = _case(n, k, e, 0.2)
    x, w = normal(9, n, h).cuda(), normal(10, n, k).cuda()
    rows = B.moe_dispatch(x, g, k)
    dy = normal(11, n, h).cuda()
    drows, dw = B.moe_combine_backward(dy, rows, w, g)
    dx = B.moe_dispatch_backward(drows, g, k)

    def loss(x, w):
        y = B.moe_combine(B.moe_dispatch(x, g, k), w, g)
        return float((y.double() * dy.double()).sum())

    ux, uw = normal(12, n, h).cuda(), normal(13, n, k).cuda()
    by_x = (loss(x + ux, w) - loss(x - ux, w)) / 2
    by_w = (loss(x, w + uw) - loss(x, w - uw)) / 2
    want_x = float((dx.double() * ux.double()).sum())
    want_w = float((dw.double() * uw.double()).sum())
    mag_x = float((dx.abs().double() * ux.abs().double()).sum())
    mag_w = float((dw.abs().double() * uw.abs().double()).sum())
    rows_mag = float((drows.abs().double() * rows.abs().double()).sum())
    tol = 2.0 ** -18 * (rows_mag + mag_x + mag_w)
    assert abs(by_x - want_x) <= tol, (by_x, want_x)
    assert abs(by_w - want_w) <= tol, (by_w, want_w)


def test_combine_into_its_base():
    n, k, e, h = 9, 2, 4, 100
    _, _, g = _case(n, k, e, 0.0)
    rows, w, y = normal(1, n * k, h).cuda(), normal(2, n, k).cuda(), normal(3, n, h).cuda()
    want = B.moe_combine(rows, w, g, base=y)
    assert want is not y
    got = B.moe_combine(rows, w, g, base=y, y=y)
    assert got is y and torch.equal(got, want)


def test_groupings_of_moe_group_and_no_tokens():
    ids = torch.from_numpy(make_ids(50, 4, 16, 0.3, seed=3)).cuda()
    g = B.moe_group(ids, 16)
    x = normal(1, 50, 96, dtype=BF16).cuda()
    rows = B.moe_dispatch(x, g, 4)
    total = int(g[1][-1])
    assert torch.equal(rows[:total], x[(g[2][:total] // 4).long()])
    assert not rows[total:].any()
    g0 = B.moe_group(ids[:0], 16)
    assert B.moe_dispatch(x[:0], g0, 4).shape == (0, 96)
    assert B.moe_dispatch_backward(rows[:0], g0, 4).shape == (0, 96)
    w0 = torch.zeros(0, 4, device="cuda")
    assert B.moe_combine(rows[:0], w0, g0).shape == (0, 96)
    drows, dw = B.moe_combine_backward(x[:0], rows[:0], w0, g0)
    assert drows.shape == (0, 96) and dw.shape == (0, 4)


def test_rows_past_32_bit_offsets():
    # rows 2.2 million elements apart: the last of 1030 starts past 2^31 elements
    n, k, h, stride = 515, 2, 40, 2_200_000
    ids, (_, off, perm, inv), g = _case(n, k, 8, 0.0)
    assert (n * k - 1) * stride > 2 ** 31
    buf = torch.empty((n * k, stride), dtype=BF16, device="cuda")
    x = normal(1, n, h, dtype=BF16).cuda()
    rows = B.moe_dispatch(x, g, k, rows=buf[:, :h])
    assert torch.equal(rows.cpu(), x.cpu()[torch.from_numpy(perm).long() // k])
    w = torch.ones(n, k, device="cuda")
    y = B.moe_combine(rows, w, g)
    assert torch.equal(y, B.moe_dispatch_backward(rows, g, k))
    assert torch.equal(y, x * 2)
    drows, dw = B.moe_combine_backward(x, rows, w, g, drows=buf[:, 64:64 + h])
    assert torch.equal(drows, rows)
    del buf, rows, drows
    torch.cuda.empty_cache()


def test_calls_on_another_stream_and_in_a_graph():
    n, k, e, h = 64, 6, 32, 512
    _, _, g = _case(n, k, e, 0.1)
    x, w = normal(1, n, h, dtype=BF16).cuda(), normal(2, n, k).cuda()
    logits, dwr = normal(3, n, e).cuda(), normal(4, n, k).cuda()
    ids = torch.topk(logits, k, dim=1).indices.int().contiguous()

    def passes(stream=None):
        rows = B.moe_dispatch(x, g, k, stream=stream)
        y = B.moe_combine(rows, w, g, base=x, stream=stream)
        drows, dw = B.moe_combine_backward(y, rows, w, g, stream=stream)
        dx = B.moe_dispatch_backward(drows, g, k, stream=stream)
        dl = B.moe_route_backward(logits, ids, dwr, stream=stream)
        return rows, y, drows, dw, dx, dl

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
        x.add_(1)
        want = [t.clone() for t in passes()]
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


@pytest.mark.parametrize("n,e,k,spread", [(1, 1, 1, 1.0), (1, 256, 6, 1.0), (3, 5, 5, 3.0),
                                          (13, 101, 3, 1.5), (130, 64, 8, 10.0),
                                          (9, 1024, 8, 30.0), (50, 65, 2, 0.1),
                                          (21, 63, 4, 250.0)])
def test_route_backward(n, e, k, spread):
    # fp64 throughout (relative 2^-45 covers its chain of some twenty
    # operations on terms of either sign), then one rounding to fp32
    print("case route_backward", n, e, k, spread, flush=True)
    logits, dw = (normal(1, n, e) * spread), normal(2, n, k)
    ids = torch.topk(logits, k, dim=1).indices.int()
    dl = torch.full((n, e), float("nan"), device="cuda")
    B.moe_route_backward(logits.cuda(), ids.contiguous().cuda(), dw.cuda(), 1.5, dlogits=dl)
    ref = route_backward_ref(logits.numpy(), ids.numpy(), dw.numpy(), 1.5)
    mag = np.abs(ref).max(axis=1, keepdims=True)
    assert_within(dl, ref, U32 * np.abs(ref) + 2.0 ** -45 * mag + 2.0 ** -149, "dlogits")
    if k == 1:
        assert not dl.any()


def test_route_backward_matches_differences_of_the_router():
    # central differences of the routed weights (64 bits, the definition):
    # error of third order in a step of 1e-4, and 2^-24 of the result
    n, e, k, scale = 6, 24, 4, 1.5
    logits, dw = normal(3, n, e), normal(4, n, k)
    ids, w = B.moe_route(logits.cuda(), k, scale)
    dl = B.moe_route_backward(logits.cuda(), ids, dw.cuda(), scale).cpu().double().numpy()
    ids, l = ids.cpu().numpy(), logits.double().numpy()

    def loss(l):
        s = np.sqrt(np.logaddexp(0, np.take_along_axis(l, ids.astype(np.int64), 1)))
        return float((scale * s / s.sum(1, keepdims=True) * dw.double().numpy()).sum())

    assert abs(float((w.cpu().double() * dw.double()).sum()) - loss(l)) <= 24 * 4 * U32
    for t in range(n):
        for c in range(e):
            up, dn = l.copy(), l.copy()
            up[t, c] += 1e-4
            dn[t, c] -= 1e-4
            assert abs((loss(up) - loss(dn)) / 2e-4 - dl[t, c]) <= 1e-6


def test_route_backward_far_logits_and_left_out_slots():
    e, k = 40, 4
    # all of a token's logits far below zero (softplus is e^l there), far above,
    # or of both kinds
    l = torch.zeros(4, e)
    l[0, :k] = torch.tensor([-50.0, -60.0, -55.5, -300.0])
    l[1, :k] = torch.tensor([80.0, 1000.0, 3e4, 90.0])
    l[2, :k] = torch.tensor([-45.0, 30.0, 0.0, -700.0])
    l[3, :k] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    ids = torch.arange(k, dtype=torch.int32).repeat(4, 1)
    ids[3, 1] = -1
    dw = normal(5, 4, k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl = B.moe_route_backward(l.cuda(), ids.cuda(), dw.cuda(), 1.5, dev_error=err)
    ref = route_backward_ref(l.numpy(), ids.numpy(), dw.numpy(), 1.5)
    mag = np.abs(ref).max(axis=1, keepdims=True)
    assert_within(dl, ref, U32 * np.abs(ref) + 2.0 ** -45 * mag + 2.0 ** -149, "dlogits")
    assert int(err) == 0
    ids[2, 0], ids[1, 3] = e, -7
    dl = B.moe_route_backward(l.cuda(), ids.cuda(), dw.cuda(), 1.5, dev_error=err)
    ref = route_backward_ref(l.numpy(), ids.numpy(), dw.numpy(), 1.5)
    assert_within(dl, ref, U32 * np.abs(ref) + 2.0 ** -45 * np.abs(ref).max(1, keepdims=True)
                  + 2.0 ** -149, "dlogits")
    assert int(err) == B.MOE_DEVERR_EXPERT_ID
    all_out = B.moe_route_backward(l.cuda(), torch.full_like(ids, -1).cuda(), dw.cuda(), 1.5)
    assert not all_out.any()


@pytest.mark.parametrize("keep_max,min_w", [(4, 0.0), (0, 0.24), (3, 0.26), (1, 0.0)])
def test_gradient_of_pruned_weights_by_way_of_the_unpruned_routing(keep_max, min_w):
    # Against central differences of the definition in 64 bits with the kept
    # slots held (third order in a step of 1e-4: below 1e-7).  w, and so alpha, G
    # and dw, carry a few steps of 2^-24 each: some 10 on values of up to 8,
    # of which the router's gradient keeps less than a half: 3e-6.
    n, e, k, scale = 8, 24, 6, 1.5
    logits, g = normal(21, n, e), normal(22, n, k)
    ids, w = B.moe_route(logits.cuda(), k, scale)
    pids, pw = B.moe_route_ex(logits.cuda(), k, B.make_opts(keep_max=keep_max, min_w=min_w), scale)
    kept = pids >= 0
    assert torch.equal(pids[kept], ids[kept]) and 0 < int(kept.sum()) < n * k
    w64, g64 = w.double(), g.cuda().double()
    a = w64.square().sum(1, keepdim=True)
    kk = (w64.square() * kept).sum(1, keepdim=True)
    alpha = (a / kk).sqrt()
    big_g = (g64 * w64 * kept).sum(1, keepdim=True)
    dw = alpha * (g64 * kept + big_g * w64 * (1 / a - kept / kk))
    dl = B.moe_route_backward(logits.cuda(), ids, dw.float(), scale).cpu().double().numpy()

    ids, kept, l = ids.cpu().numpy().astype(np.int64), kept.cpu().numpy(), logits.double().numpy()

    def pruned(l):
        s = np.sqrt(np.logaddexp(0, np.take_along_axis(l, ids, 1)))
        w = scale * s / s.sum(1, keepdims=True)
        return w * kept * np.sqrt((w * w).sum(1, keepdims=True)
                                  / (w * w * kept).sum(1, keepdims=True))

    assert np.abs(pruned(l) - pw.cpu().double().numpy()).max() <= 8 * U32 * scale * 6 ** 0.5
    for c in range(e):
        up, dn = l.copy(), l.copy()
        up[:, c] += 1e-4
        dn[:, c] -= 1e-4
        diff = ((pruned(up) - pruned(dn)) * g.double().numpy()).sum(1) / 2e-4
        assert np.abs(diff - dl[:, c]).max() <= 3e-6, c


# 2048 tokens and more: 256 threads a token at most, several rounds of columns
# for each (bf16 above 2048 columns, fp32 above 1024), aligned rows and others.
# The references are taken in 64 bits on the GPU.
@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("n,k,e,h,drop,pad", [
    (2048, 2, 16, 4096, 0.0, 0), (2049, 3, 37, 2059, 0.2, 1), (2500, 1, 8, 4104, 0.0, 0),
    (2047, 2, 16, 4096, 0.1, 0), (4097, 6, 64, 1032, 0.1, 0), (2048, 8, 256, 5003, 0.3, 3)])
def test_combine_backward_of_large_batches(n, k, e, h, drop, pad, dtype, y_dtype):
    print("case combine_backward large", n, k, e, h, drop, pad, dtype, y_dtype, flush=True)
    ids, (_, off, perm, inv), g = _case(n, k, e, drop)
    total = int(off[-1])
    gen = torch.Generator(device="cuda").manual_seed(n + h)
    rows, dy, w = (torch.randn(*shape, generator=gen, device="cuda").to(t) for shape, t in
                   (((n * k, h), dtype), ((n, h), y_dtype), ((n, k), F32)))
    rows[total:] = float("nan")
    rows, dy = strided(rows, pad), strided(dy, pad)
    drows, dw = B.moe_combine_backward(dy, rows, w, g)
    f = g[2][:total].long()
    ref = w.view(-1)[f, None].double() * dy[f // k].double()
    over = (drows[:total].double() - ref).abs() - ref.abs() * (U32 + half_step(dtype) * (1 + U32))
    assert float(over.max()) <= 0
    assert not drows[total:].any()
    terms = dy[f // k].double() * rows[:total].double()
    chain = 8 * -(-h // 1024) + 10  # a lane's columns, six steps over the lanes, four wavefronts
    over = (dw.view(-1)[f].double() - terms.sum(1)).abs() - chain * U32 * terms.abs().sum(1)
    assert float(over.max()) <= 0
    dropped = torch.from_numpy(inv < 0).cuda()
    assert not dw.view(-1)[dropped].any()
    again = B.moe_combine_backward(dy, rows, w, g)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)


def test_autograd_records_nothing():
    n, k, e, h = 5, 2, 4, 24
    _, _, g = _case(n, k, e, 0.0)
    x, w = (normal(i, n, c).cuda().requires_grad_() for i, c in ((1, h), (2, k)))
    rows = B.moe_dispatch(x, g, k)
    y = B.moe_combine(rows, w, g, base=x)
    for t in (rows, y, B.moe_dispatch_backward(rows, g, k)) + B.moe_combine_backward(y, rows, w, g):
        assert not t.requires_grad and t.grad_fn is None
