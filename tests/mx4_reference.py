"""A plain float64 implementation of the microscaled 4-bit format, written from
its definition with numpy and no use of the library; the tests of the 4-bit
operators compare against it."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes, scales) of a float64 array of rows, as the format defines them."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    nb = -(-K // 32)
    codes = np.zeros((rows, nb * 32), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        v = x[:, 32 * b:32 * b + 32]
        bad = ~np.isfinite(v).all(axis=1)
        top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0)).max(axis=1))
        e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127).clip(-127, 127)
        a = np.ldexp(np.abs(np.where(bad[:, None], 0.0, v)), -e[:, None])
        lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
        hi = np.minimum(lo + 1, 7)
        below, above = a - GRID[lo], GRID[hi] - a
        c = np.where(above < below, hi, np.where(above > below, lo, np.where(lo % 2 == 0, lo, hi)))
        c = np.where(a >= 6, 7, c)
        codes[:, 32 * b:32 * b + v.shape[1]] = np.where(bad[:, None], 0, c + 8 * np.signbit(v)).astype(np.uint8)
        scales[:, b] = np.where(bad, 255, e + 127)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return packed[:, :(K + 1) // 2].copy(), scales


def values(codes, scales, K):
    """The float64 values that codes and scales stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.empty((codes.shape[0], 2 * codes.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    c = c[:, :K]
    s = np.repeat(scales.astype(np.int64), 32, axis=1)[:, :K]
    v = np.ldexp(GRID[c & 7], s - 127) * np.where(c >= 8, -1.0, 1.0)
    return np.where(s == 255, np.nan, v)
