"""Microscaled 8-bit rows, the root-mean-square norm and its gradients in 64 bits,
from the definitions (numpy): the plain implementation that the kernels are
tested against."""
import numpy as np

BLOCK = 32
# magnitudes of the codes 0 .. 126 (127 is NaN)
GRID = np.array([(m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                 for e in range(16) for m in range(8)][:127])


def nearest_code(a):
    """Code of the grid value nearest to magnitude a, ties to the even code."""
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    down, up = a - GRID[lo], GRID[hi] - a
    return np.where((hi > lo) & ((up < down) | ((up == down) & (hi % 2 == 0))), hi, lo)


def exponent(amax):
    """The least e of at least -127 with amax <= 448 * 2^e."""
    m, ex = np.frexp(np.where(amax > 0, amax, 1.0))
    e = ex - 9 + (m > 0.875)
    return np.where(amax > 0, np.maximum(e, -127), -127)


def quantize(x):
    """(codes, scales): uint8 [R, 32*nb] and [R, nb] of a float64 matrix."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nb = -(-K // BLOCK)
    b = np.zeros((R, nb * BLOCK))
    b[:, :K] = x
    b = b.reshape(R, nb, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = exponent(np.abs(b).max(-1))
    code = nearest_code(np.abs(b) / np.exp2(e.astype(float))[..., None])
    code = (code + 128 * np.signbit(b)).astype(np.uint8)
    code[bad] = 0
    return code.reshape(R, -1), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes, scales):
    """float64 [R, 32*nb] of codes and scales (NaN where the scale is 255 or
    the code is NaN's)."""
    grid = np.append(GRID, np.nan)
    v = np.where(codes >= 128, -1.0, 1.0) * grid[codes & 127]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def norm(h, g, eps):
    """(y, rstd) of the rows of h."""
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * g, rstd


def norm_gradients(dy, h, g, rstd, dh=None):
    """(dx, dg, magnitudes that their rounding errors scale with)."""
    n = h * rstd[:, None]
    c = (dy * g * n).mean(1, keepdims=True)
    dx = rstd[:, None] * (dy * g - n * c)
    size = rstd[:, None] * (np.abs(dy * g) + np.abs(n) * np.abs(dy * g * n).mean(1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, (dy * n).sum(0), size, np.abs(dy * n).sum(0)
