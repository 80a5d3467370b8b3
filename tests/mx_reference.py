"""Microscaled 4-bit values in 64 bits, from the definition (numpy): the plain
implementation that the kernels are tested against."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = 32


def nearest_code(a):
    """Code of the grid value nearest to magnitude a, ties to the even code."""
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    down, up = a - GRID[lo], GRID[hi] - a
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(take_hi & (hi > lo) & (a < 6), hi, lo)


def quantize(x):
    """(codes, scales): uint8 [R, 16*nb] and [R, nb] of a float64 matrix."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nb = -(-K // BLOCK)
    b = np.zeros((R, nb * BLOCK))
    b[:, :K] = x
    b = b.reshape(R, nb, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2
    e = np.where(amax > 0, np.maximum(e, -127), -127)
    code = nearest_code(np.abs(b) / np.exp2(e.astype(float))[..., None])
    code = (code + 8 * np.signbit(b)).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(R, -1)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """float64 [R, 32*nb] of codes and scales (NaN where the scale is 255)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def product(alpha, a, b, beta=0.0, c=None):
    """alpha*A*B^T + beta*C of float64 values, and the magnitude its rounding
    errors scale with."""
    r = alpha * (a @ b.T)
    t = abs(alpha) * (np.abs(a) @ np.abs(b).T)
    if beta:
        r, t = r + beta * c, t + np.abs(beta * c)
    return r, t
