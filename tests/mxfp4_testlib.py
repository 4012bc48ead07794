"""64-bit references of the MXFP4 rows, their products and the RMS norm."""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BORDERS = (E2M1[1:] + E2M1[:-1]) / 2
SIGNED = np.concatenate([E2M1, -E2M1])


def quantize_ref(x):
    """(codes uint8 [n][c/2], scale bytes uint8 [n][c/32]) of fp64 rows."""
    n, c = x.shape
    b = x.reshape(n, c // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    a = np.abs(np.where(finite[..., None], b, 0)).max(axis=2)
    e = np.frexp(np.maximum(a, 2.0 ** -130))[1] - 1  # floor(log2 a)
    byte = np.clip(e - 2, -125, 125) + 127
    v = np.where(finite[..., None], b, 0) / np.exp2(byte - 127.0)[..., None]
    m = np.abs(v)
    # the first value whose upper border is not below m; on a border the even one
    code = np.searchsorted(BORDERS, m.reshape(-1), side="left").reshape(m.shape)
    tie = (code < 7) & (m == BORDERS[np.minimum(code, 6)]) & (code % 2 == 1)
    code = code + tie + 8 * np.signbit(v)
    code = np.where(finite[..., None], code, 0).reshape(n, c).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(finite, byte, 255).astype(np.uint8)


def values(codes, scales):
    """fp64 values of codes [..][c/2] under scale bytes [..][c/32]."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return SIGNED[code] * np.repeat(s, 32, axis=-1)


def scale_words(scales):
    """Scale bytes [..][n][c/32] as words [..][words][n][16], padded with 0."""
    *lead, n, b = scales.shape
    words = -(-b // 16)
    out = np.zeros((*lead, n, words * 16), np.uint8)
    out[..., :b] = scales
    return np.ascontiguousarray(np.swapaxes(out.reshape(*lead, n, words, 16), -3, -2))


def random_mxfp4(seed, *shape, mid=127, spread=2):
    """Codes [..][c/2] and scale bytes [..][c/32] for a shape [..][c]; every
    code occurs, scales lie within 2^+-spread of 2^(mid-127)."""
    rng = np.random.default_rng(seed)
    *lead, c = shape
    codes = rng.integers(0, 256, (*lead, c // 2), dtype=np.uint8)
    scales = rng.integers(mid - spread, mid + spread + 1, (*lead, c // 32)).astype(np.uint8)
    return codes, scales


def norm_ref(s, w, eps):
    """(n, r) in fp64."""
    r = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * r * w, r


def norm_back_ref(dy, s, w, eps, dtotal=None):
    """(dx, dweight) in fp64."""
    _, r = norm_ref(s, w, eps)
    g = w * dy
    dx = r * g - s * r ** 3 * (s * g).mean(axis=1, keepdims=True)
    return dx if dtotal is None else dx + dtotal, (dy * s * r).sum(axis=0)
