"""Inputs and 64-bit references of the rows-in-expert-order calls, their
gradients and the int8 products."""

from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make_ids(n, k, e, drop=0.0, used=None, seed=0):
    """int32 [n][k], distinct within a token, a share of slots -1; `used`
    limits the experts that occur."""
    rng = np.random.default_rng(seed)
    pool = rng.permutation(e)[: used or e]
    ids = np.stack([rng.choice(pool, k, replace=False) for _ in range(n)]) if n else \
        np.zeros((0, k))
    ids = ids.astype(np.int32)
    ids[rng.random((n, k)) < drop] = -1
    return ids


def group(ids, e):
    """counts, offsets, perm, inv_perm as numpy int32 (perm's tail 0)."""
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, e, flat), kind="stable")
    total = int((flat >= 0).sum())
    counts = np.bincount(flat[flat >= 0], minlength=e).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    inv = np.full(flat.size, -1, dtype=np.int32)
    inv[order[:total]] = np.arange(total)
    perm = order.astype(np.int32)
    perm[total:] = 0
    return counts, offsets, perm, inv


def on_gpu(arrays):
    return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays)


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def strided(t, pad):
    """The same values as a view whose rows lie pad elements further apart,
    one element into its storage; the gaps hold NaN."""
    if pad == 0:
        return t
    n, c = t.shape
    buf = torch.full((n * (c + pad) + 1,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[1:].view(n, c + pad)[:, :c]
    v.copy_(t)
    return v


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound everywhere, in 64 bits on the CPU."""
    got = got.detach().double().cpu().numpy()
    ref, bound = np.asarray(ref), np.broadcast_to(np.asarray(bound), np.shape(ref))
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - ref) - bound
    if over.size and over.max() > 0:
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError("%s: %r at %s, expected %r within %r"
                             % (what, got[i], i, ref[i], bound[i]))


def route_backward_ref(logits, ids, dw, scale):
    """dlogits in 64 bits; ids outside [0, e) are left out."""
    n, e = logits.shape
    out = np.zeros((n, e))
    for t in range(n):
        at = [i for i in range(ids.shape[1]) if 0 <= ids[t, i] < e]
        if not at:
            continue
        l = logits[t, ids[t, at]].astype(np.float64)
        d = dw[t, at].astype(np.float64)
        s = np.sqrt(np.logaddexp(0.0, l))
        total = s.sum()
        slope = np.exp(-np.logaddexp(0.0, -l)) / (2 * s)
        pull = np.array([(s * (d[i] - d)).sum() for i in range(len(at))])
        out[t, ids[t, at]] = scale / total * (pull / total) * slope
    return out


def quantize_ref(x):
    """(q int8, scale fp32) of finite rows."""
    x = x.astype(np.float64)
    a = np.abs(x).max(axis=1, keepdims=True)
    q = np.rint(np.divide(x * 127, a, out=np.zeros_like(x), where=a > 0))
    return q.astype(np.int8), (a[:, 0].astype(np.float32) / np.float32(127))


def product_ref(wq, ws, q, scale, offsets, left):
    """fp64 [slots][rows] and, per output, the product; left[p]: q's row."""
    out = np.zeros((len(left), wq.shape[1]))
    for e in range(wq.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            r = left[a:b]
            acc = q[r].astype(np.float64) @ wq[e].astype(np.float64).T
            out[a:b] = acc * scale[r, None].astype(np.float64) * ws[e].astype(np.float64)
    return out


def int8_weight(seed, e, rows, cols):
    rng = np.random.default_rng(seed)
    q = rng.integers(-128, 128, (e, rows, cols), dtype=np.int8)
    scale = rng.uniform(0.5, 2.0, (e, rows)).astype(np.float32) / np.float32(74 * cols ** 0.5)
    return q, scale
