"""8-bit block-scaled operands: quantisation, RMS norm and products in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

e4m3 ("fn" form): sign, 4 exponent bits with bias 7, 3 mantissa bits; value
``(1 + m/8) 2**(e - 7)`` for ``e > 0`` and ``m/8 * 2**-6`` for ``e == 0``; codes
0x7f and 0xff are NaN, there is no infinity, and the largest value is 448.

A block of 128 consecutive columns (of one row, or of 128 rows) has the scale
``fl32(amax / 448)``, at least ``2**-126``; a value stands for ``code * scale``.
Scales are rows of one column per block, padded with zeros to a multiple of 4.
"""
from __future__ import annotations

import numpy as np

MIN_SCALE = 2.0 ** -126


def e4m3_values() -> np.ndarray:
    """fp64 value of every code."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_VALUES = e4m3_values()


def decode(codes) -> np.ndarray:
    return _VALUES[np.asarray(codes, dtype=np.uint8)]


def half_step(v) -> np.ndarray:
    """Half the spacing of e4m3 values around ``v``: the most a rounding moves it."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    return 2.0 ** (np.maximum(np.where(a > 0, e, -6.0), -6.0) - 4)


def scale_cols(k: int) -> int:
    return 4 * (-(-k // 512))


def block_scales(y, block_rows: int = 1) -> np.ndarray:
    """fp32 scales ``[ceil(rows / block_rows), scale_cols(k)]`` of ``y`` ``[rows, k]``,
    from the fp32 amax and one fp32 division."""
    y = np.asarray(y, dtype=np.float32)
    rows, k = y.shape
    out = np.zeros((-(-rows // block_rows), scale_cols(k)), dtype=np.float32)
    with np.errstate(invalid="ignore"):
        for i in range(out.shape[0]):
            for c in range(-(-k // 128)):
                amax = np.abs(y[i * block_rows:(i + 1) * block_rows, c * 128:(c + 1) * 128]).max()
                s = np.float32(amax) / np.float32(448)
                out[i, c] = np.float32(MIN_SCALE) if s < MIN_SCALE else s
    return out


def spread(scales, rows: int, k: int, block_rows: int = 1) -> np.ndarray:
    """The scale of every element, fp64 ``[rows, k]``."""
    s = np.asarray(scales, dtype=np.float64)
    return np.repeat(np.repeat(s, 128, axis=1)[:, :k], block_rows, axis=0)[:rows]


def swiglu(x) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    g, u = np.split(x, 2, axis=-1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def add_rmsnorm(x, w, r=None, eps: float = 1e-6):
    """``(h, y)`` in fp64."""
    h = np.asarray(x, dtype=np.float64)
    if r is not None:
        h = h + np.asarray(r, dtype=np.float64)
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(w, np.float64)


def mm_fp8_block(a, sa, b, sb):
    """``(out, magnitude)`` fp64 ``[m, n]`` of codes ``a``, ``b`` and their scales;
    magnitude is the sum of the absolute values of the terms."""
    (m, k), n = a.shape, b.shape[0]
    x = decode(a) * spread(sa, m, k)
    w = decode(b) * spread(sb, n, k, 128)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def group_maxima(a, sa, b, sb):
    """``[m, n]``: over every 8 consecutive k, the largest |a| of the row times the
    largest |b| of the column (at least the largest product), summed."""
    (m, k), n = a.shape, b.shape[0]
    x = np.abs(decode(a) * spread(sa, m, k)).reshape(m, k // 8, 8).max(axis=2)
    w = np.abs(decode(b) * spread(sb, n, k, 128)).reshape(n, k // 8, 8).max(axis=2)
    return x @ w.T


def grouped_mm_fp8_block(a, sa, b, sb, m_indptr):
    """``(out, magnitude, group maxima, written)``; bounds clamped into ``[0, rows]``."""
    m, n = a.shape[0], b.shape[1]
    out, mag, top = np.zeros((m, n)), np.zeros((m, n)), np.zeros((m, n))
    written = np.zeros(m, dtype=bool)
    for e in range(b.shape[0]):
        s = min(max(int(m_indptr[e]), 0), m)
        t = min(max(int(m_indptr[e + 1]), s), m)
        if t > s:
            out[s:t], mag[s:t] = mm_fp8_block(a[s:t], sa[s:t], b[e], sb[e])
            top[s:t] = group_maxima(a[s:t], sa[s:t], b[e], sb[e])
            written[s:t] = True
    return out, mag, top, written
