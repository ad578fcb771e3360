"""The residual norms without a GPU: refusals before anything is enqueued, and
the float64 reference gradient against differences of the reference forward."""
import numpy as np
import pytest

import linear_layer_amd as ll
from norm_reference import forward, gradient

E = ll.ERR_INVALID_VALUE
FINE = (ll.OK, ll.ERR_NO_DEVICE, ll.ERR_UNSUPPORTED_ARCH)
NAMES = ("Y", "w_post", "gate", "X", "w_pre", "XO", "H", "DXO", "DH", "DY", "DX", "dgate", "dw_post", "dw_pre", "ws")
P = {n: 0x10000000 * (i + 1) for i, n in enumerate(NAMES)}   # addresses nothing may touch


def fwd(M=4, N=64, type=0, ld=None, eps=1e-5, alpha=1.0, **k):
    p = {**P, **{n: v for n, v in k.items() if n in P}}
    lds = {n: k.get("ld" + n, max(N, 1) if ld is None else ld) for n in ("Y", "X", "XO", "H")}
    return ll.load().rmsnorm_residual(M, N, type, p["Y"], lds["Y"], p["w_post"], p["gate"], alpha, p["X"], lds["X"],
                                      p["w_pre"], eps, p["XO"], lds["XO"], p["H"], lds["H"], None)


def bwd(M=4, N=64, type=0, ld=None, eps=1e-5, alpha=1.0, ws_bytes=1 << 20, **k):
    p = {**P, **{n: v for n, v in k.items() if n in P}}
    lds = {n: k.get("ld" + n, max(N, 1) if ld is None else ld) for n in ("Y", "X", "DXO", "DH", "DY", "DX")}
    return ll.load().rmsnorm_residual_grad(M, N, type, p["DXO"], lds["DXO"], p["DH"], lds["DH"], p["Y"], lds["Y"],
                                           p["w_post"], p["gate"], alpha, p["X"], lds["X"], p["w_pre"], eps, p["DY"],
                                           lds["DY"], p["DX"], lds["DX"], p["dgate"], p["dw_post"], p["dw_pre"],
                                           p["ws"], ws_bytes, None)


def no_device():
    import torch
    return not torch.cuda.is_available()


def test_forward_refusals():
    assert fwd(M=-1) == E and fwd(N=-1) == E and fwd(type=3) == E and fwd(ld=63) == E
    assert fwd(eps=-1e-6) == E and fwd(eps=float("nan")) == E and fwd(eps=float("inf")) == E
    assert fwd(X=None) == E and fwd(XO=None, H=None) == E
    for n in ("Y", "X", "XO", "H", "w_post", "gate", "w_pre"):
        assert fwd(**{n: P[n] + 2}) == E
        if n not in ("XO", "H"):
            assert fwd(H=P[n]) == E
    for n in ("Y", "w_post", "gate", "w_pre", "H"):
        assert fwd(XO=P[n]) == E
    assert fwd(XO=P["X"] + 16) == E and fwd(XO=P["X"], ldXO=65) == E      # over x, but not in place
    assert fwd(type=1, X=P["X"] + 1) == E
    assert fwd(M=0, X=None, XO=None, H=None) == ll.OK and fwd(N=0, X=None) == ll.OK


def test_gradient_refusals():
    assert bwd(M=-1) == E and bwd(N=-1) == E and bwd(type=3) == E and bwd(ld=63) == E
    assert bwd(eps=-1e-6) == E and bwd(eps=float("nan")) == E
    assert bwd(X=None) == E and bwd(DXO=None, DH=None) == E
    assert bwd(Y=None) == E and bwd(Y=None, DY=None) == E and bwd(Y=None, DY=None, dgate=None) == E
    need = ll.rmsnorm_grad_workspace_size(4, 64)
    assert need == 4 * 2 * 64 * 4
    assert bwd(ws=None) == E and bwd(ws_bytes=need - 1) == E and bwd(ws_bytes=-1) == E and bwd(ws=P["ws"] + 4) == E
    outs = ("DY", "DX", "dgate", "dw_post", "dw_pre", "ws")
    for n in ("Y", "w_post", "gate", "X", "w_pre", "DH"):
        for o in outs:
            assert bwd(**{o: P[n]}) == E, (o, n)
    for o in ("DY", "dgate", "dw_post", "dw_pre", "ws"):
        assert bwd(**{o: P["DXO"]}) == E
        assert bwd(**{o: P["DX"]}) == E
    assert bwd(DX=P["DXO"] + 16) == E and bwd(DX=P["DXO"], ldDX=65) == E
    for n in outs[:5]:
        assert bwd(**{n: P[n] + 2}) == E
    assert bwd(N=0, X=None) == ll.OK


def test_good_arguments_reach_the_device_check():
    if not no_device():
        pytest.skip("a device is visible")
    assert fwd() in FINE and fwd(XO=P["X"]) in FINE and fwd(Y=None, w_post=None, gate=None, w_pre=None) in FINE
    assert fwd(H=None) in FINE and fwd(XO=None) in FINE
    assert bwd() in FINE and bwd(DX=P["DXO"]) in FINE and bwd(DH=None) in FINE
    assert bwd(Y=None, DY=None, dgate=None, dw_post=None) in FINE
    assert bwd(M=0, X=None, DXO=None, DH=None, Y=None, DY=None, DX=None, ws=None, ws_bytes=0) in FINE


def test_workspace_sizes():
    size = ll.rmsnorm_grad_workspace_size
    assert size(0, 5) == 0 and size(5, 0) == 0
    assert size(512, 4096) == size(100000, 4096) == 8 * 512 * 4096
    assert size(1, 20000) == 256 + 8 * 20000
    with pytest.raises(ValueError):
        size(-1, 4)


def test_reference_gradient_against_differences():
    """Central differences of L = <dxo, x'> + <dh, h> in float64: the step 1e-5
    leaves a truncation error near 1e-10 and a rounding error near 1e-10."""
    r = np.random.default_rng(3)
    M, N, eps, alpha = 3, 7, 1e-3, 0.6
    a = {"y": r.standard_normal((M, N)), "x": r.standard_normal((M, N)), "w_post": r.standard_normal(N),
         "gate": r.standard_normal(N), "w_pre": r.standard_normal(N)}
    dxo, dh = r.standard_normal((M, N)), r.standard_normal((M, N))

    def loss(v):
        xo, h, _, _ = forward(v["y"], v["x"], v["w_post"], v["gate"], alpha, v["w_pre"], eps)
        return (dxo * xo).sum() + (dh * h).sum()

    g = gradient(dxo, dh, a["y"], a["x"], a["w_post"], a["gate"], alpha, a["w_pre"], eps)
    for name, out in (("y", "dy"), ("x", "dx"), ("gate", "dgate"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        for i in np.ndindex(a[name].shape):
            up, down = ({**a, name: a[name].copy()} for _ in range(2))
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - g[out][0][i]) < 1e-7, (name, i)
