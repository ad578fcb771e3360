"""The 16-bit layer, its gradients and the microscaled 8-bit format in float64, from
their definitions, with numpy and no use of the library. Sums come with the sum
of their terms' magnitudes, which is what rounding errors scale with."""
import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def _decode_table():
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if c & 127 == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        t[c] = -v if c & 128 else v
    return t


TABLE = _decode_table()
POSITIVE = TABLE[:127]   # ascending


def mx8_quantize(x):
    """(codes, scales) of a float64 array of rows."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    codes, scales = np.zeros((rows, K), np.uint8), np.zeros((rows, -(-K // 32)), np.uint8)
    for b in range(scales.shape[1]):
        v = x[:, 32 * b:32 * b + 32]
        for r in range(rows):
            if not np.isfinite(v[r]).all():
                scales[r, b] = 255
                continue
            top, e = np.abs(v[r]).max(initial=0.0), -127
            while top > 448 * 2.0 ** e:
                e += 1
            scales[r, b] = e + 127
            a = np.abs(v[r]) / 2.0 ** e
            hi = np.searchsorted(POSITIVE, a).clip(1, 126)
            lo = hi - 1
            dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
            c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
            codes[r, 32 * b:32 * b + 32] = c | np.where(np.signbit(v[r]), 128, 0)
    return codes, scales


def mx8_values(codes, scales):
    s = np.repeat(scales.astype(np.int64), 32, axis=1)[:, :codes.shape[1]]
    return np.where(s == 255, math.nan, TABLE[codes] * 2.0 ** (s - 127.0))


def act(z, kind):
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(z, kind):
    if kind == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if kind == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def bounds(offsets, M):
    """(begin, end) of each group: offsets held to 0 .. M, none below its predecessor."""
    if offsets is None:
        return [(0, M)]
    b = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M))
    return list(zip(b[:-1].tolist(), b[1:].tolist()))


def linear(x, w, bias, spans):
    """(z, size of z), nan in the rows of no group; w, bias stacked by group."""
    z = np.full((x.shape[0], w.shape[1]), math.nan)
    t = z.copy()
    for g, (a, e) in enumerate(spans):
        z[a:e], t[a:e] = x[a:e] @ w[g].T, np.abs(x[a:e]) @ np.abs(w[g]).T
        if bias is not None:
            z[a:e] += bias[g]
            t[a:e] += np.abs(bias[g])
    return z, t


def grad_input(dz, w, spans):
    dx = np.full((dz.shape[0], w.shape[2]), math.nan)
    t = dx.copy()
    for g, (a, e) in enumerate(spans):
        dx[a:e], t[a:e] = dz[a:e] @ w[g], np.abs(dz[a:e]) @ np.abs(w[g])
    return dx, t


def grad_weight(dz, x, spans):
    return (np.stack([dz[a:e].T @ x[a:e] for a, e in spans]),
            np.stack([np.abs(dz[a:e]).T @ np.abs(x[a:e]) for a, e in spans]))
