"""Block-scaled FP8 in plain fp64: E4M3 codes with a power-of-two scale for
each 128 values of a row, or each 128 x 128 block of a weight matrix, and the
layer, its weight gradient and the GELU's slope on the values they hold.

(The pages have no counterpart: the format is OCP E4M3FN with E8M0 scales,
the scale the smallest power of two that brings a block's largest finite
magnitude to at most 448, and at least 2^-117.)"""

import numpy as np
from scipy.special import erfc

from .qlinear import e4m3_round

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE_EXP = -117


def fp8_scale_exponent(amax):
    """e with 2^e the scale of a block whose largest finite magnitude is amax."""
    e = MIN_SCALE_EXP
    while amax / 2.0 ** e > E4M3_MAX:
        e += 1
    return e


def fp8_encode(x, rows=1):
    """(code values, scale exponents) of x [n, d], a scale per rows x 128 block.
    The code of a value that is not finite is NaN."""
    x = np.asarray(x, dtype=np.float64)
    n, d = x.shape
    q = np.empty_like(x)
    exps = np.empty((-(-n // rows), -(-d // BLOCK)), dtype=np.int64)
    for i in range(exps.shape[0]):
        for j in range(exps.shape[1]):
            at = np.s_[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            b = x[at]
            fin = np.isfinite(b)
            exps[i, j] = e = fp8_scale_exponent(np.max(np.abs(b[fin]), initial=0.0))
            q[at] = np.where(fin, e4m3_round(np.where(fin, b, 0.0) / 2.0 ** e), np.nan)
    return q, exps


def fp8_scales(exps, rows, shape):
    """The scale of every element of a matrix of this shape."""
    s = np.ldexp(1.0, exps)
    return np.repeat(np.repeat(s, rows, 0)[:shape[0]], BLOCK, 1)[:, :shape[1]]


def fp8_decode(q, exps, rows=1):
    return q * fp8_scales(exps, rows, q.shape)


def normal_cdf(x):
    return 0.5 * erfc(-x / np.sqrt(2.0))


def gelu_slope(x):
    """d/dx x Phi(x) = Phi(x) + x phi(x)."""
    return normal_cdf(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
