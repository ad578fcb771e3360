"""The residual step and its gradient in float64, from their formulas, with
numpy and no use of the library. Each function also gives the size of every
result: the same expression with every term's magnitude added, which is what
rounding errors scale with."""
import numpy as np


def _r(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def forward(y, x, w_post, gate, alpha, w_pre, eps):
    """(x', h, size of x', size of h)."""
    if y is None:
        xo, size = x, np.abs(x)
    else:
        step = alpha * gate * (y * _r(y, eps) * w_post)
        xo, size = x + step, np.abs(x) + np.abs(step)
    rx = _r(xo, eps)
    return xo, xo * rx * w_pre, size, size * rx * np.abs(w_pre)


def gradient(dxo, dh, y, x, w_post, gate, alpha, w_pre, eps):
    """{name: (value, size)} for dy, dx, dgate, dw_post, dw_pre."""
    t = alpha * gate * w_post
    ry = _r(y, eps)
    u = y * ry
    xo, _, sxo, _ = forward(y, x, w_post, gate, alpha, w_pre, eps)
    rx = _r(xo, eps)
    n, sn = xo * rx, sxo * rx
    k = dh * w_pre
    total = dxo + rx * (k - n * (k * n).mean(axis=1, keepdims=True))
    st = np.abs(dxo) + rx * (np.abs(k) + sn * (np.abs(k) * sn).mean(axis=1, keepdims=True))
    c, sc = total * t, st * np.abs(t)
    au = np.abs(u)
    dy = ry * (c - u * (c * u).mean(axis=1, keepdims=True))
    sdy = ry * (sc + au * (sc * au).mean(axis=1, keepdims=True))
    s, ss = (total * u).sum(axis=0), (st * au).sum(axis=0)
    return {"dy": (dy, sdy), "dx": (total, st), "dgate": (alpha * w_post * s, abs(alpha) * np.abs(w_post) * ss),
            "dw_post": (alpha * gate * s, abs(alpha) * np.abs(gate) * ss),
            "dw_pre": ((dh * n).sum(axis=0), (np.abs(dh) * sn).sum(axis=0))}
