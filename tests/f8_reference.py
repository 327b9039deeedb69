"""The 8-bit block format from its definition, in float64 (numpy)."""

import numpy as np

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LEAST_EXP = {"e4m3": -6, "e5m2": -14}


def up(x, m):
    return -(-x // m) * m


def code_values(fmt):
    """float64 [256]: what each byte stands for (sign, exponent, mantissa)."""
    b = np.arange(256)
    mb = MANTISSA[fmt]
    bias = 7 if fmt == "e4m3" else 15
    sign = np.where(b & 0x80, -1.0, 1.0)
    e = (b & 0x7F) >> mb
    m = (b & 0x7F) & ((1 << mb) - 1)
    v = np.where(e == 0, m * 2.0 ** (1 - bias - mb), (1 + m / 2.0 ** mb) * 2.0 ** (e - float(bias)))
    if fmt == "e4m3":
        v[(b & 0x7F) == 0x7F] = np.nan
    else:
        v[(b & 0x7F) == 0x7C] = np.inf
        v[(b & 0x7F) > 0x7C] = np.nan
    return sign * v


def round_f8(v, fmt):
    """float64 values within the format's range, rounded to its grid (ties to even)."""
    _, e = np.frexp(v)
    step = 2.0 ** (np.maximum(e - 1, LEAST_EXP[fmt]) - MANTISSA[fmt])
    return np.rint(v / step) * step


def quantize(x, fmt, block_rows, transpose=False):
    """x [rows, cols] -> (values [rows, K] float64, scale bytes [R, Ks])."""
    x = np.asarray(x, dtype=np.float64)
    if transpose:
        x = x.T
    rows, cols = x.shape
    K, R = up(cols, 128), up(rows, block_rows)
    p = np.zeros((R, K))
    p[:rows, :cols] = x
    t = p.reshape(R // block_rows, block_rows, K // 128, 128)
    a = np.where(np.isfinite(t), np.abs(t), 0.0).max(axis=(1, 3))
    frac, e = np.frexp(a)   # a = frac 2^e, 1/2 <= frac < 1; the largest is 7/8 2^9 or 7/8 2^16
    e = e - (9 if fmt == "e4m3" else 16) + (frac > 0.875)
    e = np.where(a > 0, np.maximum(e, -127), 0)
    with np.errstate(invalid="ignore"):
        y = t / 2.0 ** e[:, None, :, None]
        fin = np.isfinite(y)
        q = np.where(fin, round_f8(np.where(fin, y, 0.0), fmt), np.nan)
    if fmt == "e5m2":
        q = np.where(np.isinf(t), t, q)
    s = np.full((R // block_rows, up(K // 128, 4)), 127, dtype=np.uint8)
    s[:, :K // 128] = e + 127
    return q.reshape(R, K)[:rows], s


def stand_for(q, s, block_rows):
    """The numbers that values q [rows, K] and scale bytes s stand for."""
    rows, K = q.shape
    e = s[:, :K // 128].astype(np.float64) - 127
    f = np.repeat(np.repeat(2.0 ** e, 128, axis=1), block_rows, axis=0)[:rows]
    return q * f
