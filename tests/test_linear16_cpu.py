"""The 16-bit layer, its gradients and the 8-bit format without a GPU: refusals
before anything is enqueued, sizes of workspaces, and the float64 references
against differences and closed forms."""
import numpy as np
import pytest

import linear16_reference as ref
import linear_layer_amd as ll

E = ll.ERR_INVALID_VALUE
FINE = (ll.OK, ll.ERR_NO_DEVICE, ll.ERR_UNSUPPORTED_ARCH)
NAMES = ("X", "offsets", "W", "bias", "R", "Y", "Z", "ZQ", "ZS", "DY", "DZ", "dbias", "ws", "DX", "XQ", "XS", "DW")
P = {n: 0x10000000 * (i + 1) for i, n in enumerate(NAMES)}   # addresses nothing may touch
BF16, F16, F32 = ll.TYPE_BF16, ll.TYPE_F16, ll.TYPE_F32


def has_device():
    import torch
    return torch.cuda.is_available()


def args(k, lds):
    p = {**P, **{n: v for n, v in k.items() if n in P}}
    return p, {n: k.get("ld" + n, w) for n, w in lds.items()}


def fwd(M=4, N=64, K=32, type=BF16, ytype=BF16, act=0, groups=1, stride=0, ws_bytes=0, **k):
    k.setdefault("offsets", None)
    k.setdefault("ws", None)
    p, ld = args(k, {"X": max(K, 1), "W": max(K, 1), **{n: max(N, 1) for n in ("R", "Y", "Z", "ZQ")}, "ZS": max(-(-N // 32), 1)})
    return ll.load().linear16_nt(M, N, K, type, p["X"], ld["X"], groups, p["offsets"], p["W"], ld["W"], stride, p["bias"],
                                 act, ytype, p["R"], ld["R"], p["Y"], ld["Y"], p["Z"], ld["Z"], p["ZQ"], ld["ZQ"], p["ZS"],
                                 ld["ZS"], p["ws"], ws_bytes, None)


def gact(M=4, N=64, type=BF16, ytype=BF16, act=4, groups=1, ws_bytes=1 << 20, **k):
    k.setdefault("offsets", None)
    k.setdefault("Z", None)
    p, ld = args(k, {**{n: max(N, 1) for n in ("DY", "Z", "ZQ", "DZ")}, "ZS": max(-(-N // 32), 1)})
    return ll.load().linear16_grad_act(M, N, type, act, ytype, p["DY"], ld["DY"], groups, p["offsets"], p["Z"], ld["Z"],
                                       p["ZQ"], ld["ZQ"], p["ZS"], ld["ZS"], p["DZ"], ld["DZ"], p["dbias"], p["ws"],
                                       ws_bytes, None)


def gin(M=4, N=64, K=32, type=BF16, xtype=BF16, groups=1, stride=0, ws_bytes=0, **k):
    k.setdefault("offsets", None)
    k.setdefault("ws", None)
    p, ld = args(k, {"DZ": max(N, 1), "W": max(K, 1), "DX": max(K, 1)})
    return ll.load().linear16_grad_input(M, N, K, type, p["DZ"], ld["DZ"], groups, p["offsets"], p["W"], ld["W"], stride,
                                         xtype, p["DX"], ld["DX"], p["ws"], ws_bytes, None)


def gw(M=4, N=64, K=32, type=BF16, wtype=BF16, beta=0.0, groups=1, stride=None, **k):
    k.setdefault("offsets", None)
    if "XQ" not in k:
        k.update(XQ=None, XS=None)
    p, ld = args(k, {"DZ": max(N, 1), **{n: max(K, 1) for n in ("X", "XQ", "DW")}, "XS": max(-(-K // 32), 1)})
    return ll.load().linear16_grad_weight(M, N, K, type, p["DZ"], ld["DZ"], groups, p["offsets"], p["X"], ld["X"], p["XQ"],
                                          ld["XQ"], p["XS"], ld["XS"], wtype, beta, p["DW"], ld["DW"],
                                          N * K if stride is None else stride, None)


def quant(M=4, K=64, type=F32, **k):
    p, ld = args(k, {"X": max(K, 1), "XQ": max(K, 1), "XS": max(-(-K // 32), 1)})
    return ll.load().mx8_quantize(M, K, type, p["X"], ld["X"], p["XQ"], ld["XQ"], p["XS"], ld["XS"], None)


def dequant(M=4, K=64, type=F32, **k):
    p, ld = args(k, {"Y": max(K, 1), "XQ": max(K, 1), "XS": max(-(-K // 32), 1)})
    return ll.load().mx8_dequantize(M, K, p["XQ"], ld["XQ"], p["XS"], ld["XS"], type, p["Y"], ld["Y"], None)


def refuses_common(call, wide):
    assert call(M=-1) == E and call(N=-1) == E and call(type=F32) == E and call(type=7) == E
    assert call(type=F16, **{wide: BF16}) == E and call(**{wide: 9}) == E
    assert call(groups=2) == E and call(groups=0) == E                            # no offsets: one group
    assert call(groups=-1, offsets=P["offsets"]) == E and call(groups=2, offsets=P["offsets"] + 2) == E
    assert call(groups=ll.MAX_GROUPS + 1, offsets=P["offsets"]) == E
    assert call(groups=0, offsets=P["offsets"]) == ll.OK
    big = 2 ** 31 - 1024
    assert call(M=big) == E and call(N=big, ldZ=big, ldZQ=big, ldZS=big // 32 + 1) == E


def test_forward_refusals():
    refuses_common(fwd, "ytype")
    assert fwd(K=-1) == E and fwd(act=-1) == E and fwd(act=5) == E and fwd(stride=-1) == E
    for n, w in (("X", 31), ("W", 31), ("R", 63), ("Y", 63), ("Z", 63), ("ZQ", 63), ("ZS", 1)):
        assert fwd(**{"ld" + n: w}) == E, n
    assert fwd(X=None) == E and fwd(W=None) == E and fwd(Y=None) == E and fwd(ZQ=None) == E and fwd(ZS=None) == E
    for n in ("X", "W", "R", "Y", "Z"):
        assert fwd(**{n: P[n] + 1}) == E, n
    assert fwd(bias=P["bias"] + 2) == E and fwd(ytype=F32, Y=P["Y"] + 2) == E
    for o in ("Y", "Z", "ZQ", "ZS"):
        for i in ("X", "W", "bias"):
            assert fwd(**{o: P[i]}) == E, (o, i)
        assert fwd(groups=2, offsets=P["offsets"], **{o: P["offsets"]}) == E
        if o != "Y":
            assert fwd(**{o: P["R"]}) == E and fwd(**{o: P["Y"]}) == E
    assert fwd(Y=P["R"] + 16) == E and fwd(Y=P["R"], ldY=65) == E                 # over R, but not in place
    # the last group's weight meets the output
    assert fwd(groups=3, offsets=P["offsets"], stride=4096, Y=P["W"] + 2 * 2 * 4096) == E
    assert fwd(M=0, X=None, Y=None) == ll.OK and fwd(N=0, Y=None) == ll.OK
    assert fwd(groups=2 ** 20, offsets=P["offsets"], stride=2 ** 62) == E         # a stack past the address space


def test_forward_takes():
    if has_device():
        pytest.skip("the addresses are not to be used")
    for k in ({}, {"ytype": F32}, {"type": F16, "ytype": F16}, {"R": None, "Z": None, "ZQ": None, "ZS": None, "bias": None},
              {"Y": P["R"]}, {"K": 0, "X": None, "W": None}, {"groups": 3, "offsets": P["offsets"], "stride": 4096},
              {"X": P["X"] + 2, "W": P["W"] + 2, "Y": P["Y"] + 2}):
        assert fwd(**k) in FINE, k


def test_activation_gradient_refusals():
    refuses_common(gact, "ytype")
    assert gact(act=-1) == E and gact(act=5) == E and gact(Z=P["Z"]) == E          # Z twice
    for n, w in (("DY", 63), ("ZQ", 63), ("ZS", 1), ("DZ", 63)):
        assert gact(**{"ld" + n: w}) == E, n
    assert gact(Z=P["Z"], ZQ=None, ZS=None, ldZ=63) == E
    assert gact(DY=None) == E and gact(ZQ=None, ZS=None) == E and gact(ZQ=None) == E and gact(DZ=None, dbias=None) == E
    for n in ("DY", "DZ", "dbias"):
        assert gact(**{n: P[n] + 1}) == E, n
    need = ll.linear16_grad_act_workspace_size(4, 64)
    assert need == 4 * 1 * 64
    assert gact(ws=None) == E and gact(ws_bytes=need - 1) == E and gact(ws_bytes=-1) == E and gact(ws=P["ws"] + 4) == E
    for o in ("DZ", "dbias", "ws"):
        for i in ("ZQ", "ZS"):
            assert gact(**{o: P[i]}) == E, (o, i)
        assert gact(groups=2, offsets=P["offsets"], **{o: P["offsets"]}) == E
    for o in ("dbias", "ws"):
        assert gact(**{o: P["DY"]}) == E and gact(**{o: P["DZ"]}) == E
        assert gact(Z=P["Z"], ZQ=None, ZS=None, **{o: P["Z"]}) == E
    assert gact(DZ=P["DY"] + 16) == E and gact(DZ=P["DY"], ldDZ=65) == E and gact(DZ=P["DY"], ytype=F32) == E
    assert gact(M=0, dbias=None) == ll.OK and gact(N=0) == ll.OK


def test_activation_gradient_takes():
    if has_device():
        pytest.skip("the addresses are not to be used")
    for k in ({}, {"DZ": P["DY"]}, {"Z": P["Z"], "ZQ": None, "ZS": None, "DZ": P["Z"]}, {"act": 0, "ZQ": None, "ZS": None},
              {"dbias": None, "ws": None, "ws_bytes": 0}, {"DZ": None}, {"M": 0, "DY": None, "DZ": None}):
        assert gact(**k) in FINE, k


def test_input_gradient_refusals():
    refuses_common(gin, "xtype")
    assert gin(K=-1) == E and gin(stride=-1) == E
    for n, w in (("DZ", 63), ("W", 31), ("DX", 31)):
        assert gin(**{"ld" + n: w}) == E, n
        assert gin(**{n: None}) == E and gin(**{n: P[n] + 1}) == E
    assert gin(DX=P["DZ"]) == E and gin(DX=P["W"]) == E and gin(groups=2, offsets=P["offsets"], DX=P["offsets"]) == E
    assert gin(M=0) == ll.OK and gin(K=0) == ll.OK
    if not has_device():
        assert gin() in FINE and gin(N=0, DZ=None, W=None) in FINE


def test_weight_gradient_refusals():
    refuses_common(gw, "wtype")
    assert gw(K=-1) == E and gw(stride=-1) == E and gw(XQ=P["XQ"]) == E and gw(X=None) == E
    both = {"X": None, "XQ": P["XQ"], "XS": P["XS"]}
    assert gw(**{**both, "XS": None}) == E and gw(**{**both, "XQ": None}) == E
    for n, w in (("DZ", 63), ("X", 31), ("DW", 31)):
        assert gw(**{"ld" + n: w}) == E, n
        assert gw(**{n: None}) == E and gw(**{n: P[n] + 1}) == E
    assert gw(**both, ldXQ=31) == E and gw(K=64, **both, ldXS=1) == E
    for i in ("DZ", "X"):
        assert gw(DW=P[i]) == E
    assert gw(**both, DW=P["XQ"]) == E and gw(**both, DW=P["XS"]) == E
    assert gw(groups=2, offsets=P["offsets"], DW=P["offsets"]) == E
    assert gw(groups=2, offsets=P["offsets"], stride=63 * 32 + 31) == E            # groups' results overlap
    assert gw(N=0) == ll.OK and gw(K=0) == ll.OK
    if not has_device():
        for k in ({}, both, {"M": 0, "DZ": None, "X": None}, {"groups": 2, "offsets": P["offsets"]}):
            assert gw(**k) in FINE, k


def test_format_refusals():
    for call, v in ((quant, "X"), (dequant, "Y")):
        assert call(M=-1) == E and call(K=-1) == E and call(type=3) == E
        for n, w in ((v, 63), ("XQ", 63), ("XS", 1)):
            assert call(**{"ld" + n: w}) == E and call(**{n: None}) == E, n
        assert call(**{v: P[v] + 2}) == E and call(type=F16, **{v: P[v] + 1}) == E
        assert call(**{v: P["XQ"]}) == E and call(**{v: P["XS"]}) == E
        assert call(M=0) == ll.OK and call(K=0) == ll.OK
        if not has_device():
            assert call() in FINE
    assert quant(XS=P["XQ"]) == E


def test_workspace_sizes():
    f = ll.linear16_grad_act_workspace_size
    assert f(0, 64) == 0 and f(5, 0) == 0 and f(1, 8, 4) == 4 * 8
    for M, N, g in ((1000, 64, 3), (8191, 4096, 16), (129, 1001, 1)):
        step = 64 if M * N >= 1 << 22 else 16
        assert f(M, N, g) == 4 * N * (M // step + min(M, g))
    for bad in ((-1, 8, 1), (8, -1, 1), (8, 8, -1), (8, 8, ll.MAX_GROUPS + 1), (2 ** 31, 8, 1)):
        with pytest.raises(ValueError):
            f(*bad)


def test_python_refusals():
    import torch
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        ll.linear16_nt(x, x, None, 0, None, x)                  # host tensors
    with pytest.raises(TypeError):
        ll.linear16_nt(x.float(), x, None, 0, None, x)
    with pytest.raises(TypeError):
        ll.linear16_grad_act(x, None, 0, x.float())
    with pytest.raises((ValueError, TypeError)):
        ll.mx8_quantize(x, x, x)


# ---- the references -----------------------------------------------------------

@pytest.mark.parametrize("kind", ref.ACTS)
def test_reference_slopes(kind):
    z = np.concatenate([np.linspace(-6, 6, 97) + 1e-3, [-20.0, 20.0]])
    h = 1e-6
    d = (ref.act(z + h, kind) - ref.act(z - h, kind)) / (2 * h)
    assert np.abs(d - ref.slope(z, kind)).max() < 1e-8


def test_reference_gradients_by_differences():
    r = np.random.default_rng(5)
    M, N, K, spans = 7, 5, 4, [(1, 3), (3, 3), (3, 6)]
    x, w, b, c = r.standard_normal((M, K)), r.standard_normal((3, N, K)), r.standard_normal((3, N)), r.standard_normal((M, N))
    rows = np.arange(1, 6)

    def loss(x, w, b):
        return (c[rows] * ref.act(ref.linear(x, w, b, spans)[0], "silu")[rows]).sum()

    z = ref.linear(x, w, b, spans)[0]
    dz = np.zeros((M, N))
    dz[rows] = c[rows] * ref.slope(z[rows], "silu")
    dx, dw = np.nan_to_num(ref.grad_input(dz, w, spans)[0]), ref.grad_weight(dz, x, spans)[0]
    db = np.stack([dz[a:e].sum(0) for a, e in spans])
    h = 1e-6
    for got, arg in ((dx, 0), (dw, 1), (db, 2)):
        for i in np.ndindex(got.shape):
            v = []
            for s in (h, -h):
                a = [x.copy(), w.copy(), b.copy()]
                a[arg][i] += s
                v.append(loss(*a))
            assert abs((v[0] - v[1]) / (2 * h) - got[i]) < 1e-8


def test_reference_format():
    assert ref.POSITIVE[-1] == 448 and (np.diff(ref.POSITIVE) > 0).all() and ref.POSITIVE[1] == 2.0 ** -9
    # every code is its own nearest, next to 448, which fixes the scale at 1
    rows = np.concatenate([np.full((4, 1), 448.0), ref.POSITIVE[:124].reshape(4, 31)], axis=1)
    codes, scales = ref.mx8_quantize(rows)
    assert (scales == 127).all() and (ref.TABLE[codes] == rows).all()
    # ties go to the even code; the scale takes the largest value in without clipping it
    codes, scales = ref.mx8_quantize(np.array([[448.0, 17.0, 19.0, -17.0]]))
    assert (ref.mx8_values(codes, scales) == [[448.0, 16.0, 20.0, -16.0]]).all()
    for t, e in ((448.0, 0), (448.5, 1), (1.75, -8), (1.7501, -7), (0.0, -127), (1e-45, -127), (3e38, 120)):
        assert ref.mx8_quantize(np.array([[t]]))[1][0, 0] == e + 127
    assert ref.mx8_quantize(np.array([[np.inf, 1.0]]))[1][0, 0] == 255


def test_kernel_names():
    k = ll.linear16_chosen_kernel
    assert k(0, 1, 11008, 4096) == "rows" and k(0, 64, 8, 8, aligned=False) == "rows_any" and k(0, 65, 8, 8) == "small"
    assert k(0, 640, 64, 64, groups=10) == "rows" and k(1, 1, 64, 64) == "small" and k(1, 1, 64, 64, aligned=False) == "small_any"
    assert k(0, 8192, 8192, 8192) == k(1, 8192, 8192, 8192) == k(2, 8192, 8192, 8192) == "large"
    for bad in ((3, 1, 1, 1), (-1, 1, 1, 1), (0, 0, 1, 1), (0, 1, 0, 1), (0, 1, 1, 0), (0, 1, 1, 1, 0), (0, 1, 1, 1, ll.MAX_GROUPS + 1)):
        assert k(*bad) == ""
    # sizes at the limits
    big = 2 ** 31 - 1025
    for op in (0, 1, 2):
        for m, n, kk, g in ((big, 1, 1, 1), (1, big, 1, 1), (1, 1, big, 1), (big, big, big, ll.MAX_GROUPS)):
            assert k(op, m, n, kk, g) in ("rows", "small", "large")


def test_workspaces_of_shares():
    def f(M, N, K, g=1):
        return ll.linear16_workspace_size(ll.L16_FORWARD, M, N, K, g)

    def d(M, N, K, g=1):
        return ll.linear16_workspace_size(ll.L16_GRAD_INPUT, M, N, K, g)

    assert f(1, 11008, 4096) == 0 and f(0, 64, 64) == 0 and f(500, 64, 64) == 0 and f(1, 200, 512) == 0
    assert f(8192, 8192, 8192) == 0 and d(8192, 8192, 8192) == 0 and d(16, 64, 4096) == 0 and d(16, 0, 64) == 0
    for n, M, N in ((f(33, 4096, 11008), 33, 4096), (f(130, 1024, 11008), 130, 1024), (d(16, 11008, 4096), 16, 4096)):
        assert n > 0 and n % (4 * M * N) == 0 and 2 <= n // (4 * M * N) <= 16
    for bad in ((-1, 8, 8), (8, -1, 8), (8, 8, -1), (8, 8, 8, -1), (2 ** 31, 8, 8)):
        for g in (f, d):
            with pytest.raises(ValueError):
                g(*bad)
    with pytest.raises(ValueError):
        ll.linear16_workspace_size(ll.L16_GRAD_WEIGHT, 8, 8, 8)
    for call in (fwd, gin):
        assert call(ws=P["ws"], ws_bytes=-1) == E and call(ws=P["ws"] + 4, ws_bytes=1 << 20) == E


def test_sizes_no_product_takes():
    most = 2 ** 31 - 1025
    for big in (most + 1, 2 ** 31 - 1):
        for shape in ((big, 8, 8), (8, big, 8), (8, 8, big), (big, big, big)):
            for product in (ll.L16_FORWARD, ll.L16_GRAD_INPUT, ll.L16_GRAD_WEIGHT):
                assert ll.linear16_chosen_kernel(product, *shape) == ""
            assert ll.linear16_workspace_size(ll.L16_FORWARD, *shape) == 0
            assert ll.linear16_workspace_size(ll.L16_GRAD_INPUT, *shape) == 0
    for shape in ((most, 8, 8), (8, most, 8), (8, 8, most), (most, most, most)):
        for product in (ll.L16_FORWARD, ll.L16_GRAD_INPUT, ll.L16_GRAD_WEIGHT):
            assert ll.linear16_chosen_kernel(product, *shape) != ""
        for product in (ll.L16_FORWARD, ll.L16_GRAD_INPUT):
            assert ll.linear16_workspace_size(product, *shape) in (0, 16 * 4 * 8 * 8)


def test_numbers_past_a_c_int():
    """Refused, not cut to their lower 32 bits."""
    for wide in (2 ** 31, 2 ** 32 + 64, -2 ** 32 + 64):
        for i in range(5):
            shape = [64, 64, 64, 1, 256]
            shape[i] = wide
            *shape, cus = shape
            with pytest.raises(ValueError):
                ll.linear16_chosen_kernel(ll.L16_FORWARD, *shape, num_cus=cus)
            if i < 4:
                with pytest.raises(ValueError):
                    ll.linear16_workspace_size(ll.L16_FORWARD, *shape)
            if i < 3:
                with pytest.raises(ValueError):
                    ll.linear16_grad_act_workspace_size(*(shape[:2] + shape[3:] if i < 2 else (64, 64, wide)))
        with pytest.raises(ValueError):
            ll.linear16_chosen_kernel(wide, 64, 64, 64)
        with pytest.raises(ValueError):
            ll.linear16_workspace_size(wide, 64, 64, 64)
