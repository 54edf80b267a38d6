"""e4m3 quantisation from its definition, in numpy and 64 bits (tests only)."""
import math

import numpy as np


def round_e4m3(v):
    """Magnitudes up to 448 rounded to three bits after the leading one (steps
    of 2^-9 below 2^-6), ties to even; infinities and NaN become NaN."""
    v = np.where(np.isfinite(v), v, np.nan)
    mag = np.maximum(np.abs(v), 2.0 ** -6)
    with np.errstate(invalid="ignore"):
        step = 2.0 ** (np.floor(np.log2(np.where(np.isnan(mag), 1.0, mag))) - 3)
    return np.rint(v / step) * step


def block_scale(amax):
    """The smallest power of two s >= 2^-126 with amax / s <= 448; 1 for 0."""
    if amax == 0:
        return 1.0
    e = math.frexp(amax / 448.0)
    power = e[1] - 1 if e[0] == 0.5 else e[1]
    return 2.0 ** max(power, -126)


def quantize_reference(x, block_rows):
    """(e4m3 values as float64, scales) of a float64 matrix."""
    m, k = x.shape
    scale = np.ones((-(-m // block_rows), -(-k // 128)))
    q = np.zeros_like(x)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            rs, cs = slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128)
            b = x[rs, cs]
            fin = np.abs(b[np.isfinite(b)])
            scale[i, j] = block_scale(fin.max() if fin.size else 0.0)
            q[rs, cs] = round_e4m3(b / scale[i, j])
    return q, scale


def dequantize(q, scale, block_rows):
    m, k = q.shape
    return q * np.repeat(np.repeat(scale, block_rows, 0)[:m], 128, 1)[:, :k]
