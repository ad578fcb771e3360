"""The 16-bit layer, its gradients and the 8-bit format on the GPU against float64
formulas (linear16_reference, which test_linear16_cpu checks against differences).

Tolerances. An FP32 sum of n products (exact in FP32 for 16-bit factors) takes at most n
additions, each off by at most a step, 2^-23, of the sum of the terms' magnitudes (a matrix
instruction may cut instead of rounding). An activation has a slope of at most 1.13
and is itself a few operations on values of at most 1 or |z|: 16 half-steps of FP32
of 1 + |z|. A result stored in 16 bits is off by half a step more, finfo.eps / 2 of its
value, or half its smallest subnormal. In 8 bits: half a step, 2^-4, of the value, or half
of the smallest code times the block's scale, which is at most 2 t / 448 for a block
whose largest is t."""
import numpy as np
import pytest

import linear16_reference as ref
import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACT = {k: getattr(ll, "ACT_" + k.upper()) for k in ref.ACTS}
STEP, H32 = 2.0 ** -23, 2.0 ** -24
GUARD = 7.0


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def strided(a, pad=0, shift=0):
    """a on the device, its rows `pad` further apart and `shift` elements off the allocation's
    start, inside a buffer of guards: (buffer, view)."""
    a = torch.as_tensor(a)
    guard = 0xA5 if a.dtype == torch.uint8 else GUARD
    buf = torch.full((*a.shape[:-1], shift + a.shape[-1] + pad), guard, dtype=a.dtype, device=DEV)
    v = buf[..., shift:shift + a.shape[-1]]
    v.copy_(a)
    return buf, v


def normal(r, *shape, t, scale=1.0):
    return torch.as_tensor(r.standard_normal(shape) * scale).to(TYPES[t])


def f64(t):
    return t.detach().double().cpu().numpy()


def stored(want, t):
    fi = torch.finfo(TYPES[t])
    return 0.0 if t == "f32" else fi.eps / 2 * np.abs(want) + fi.smallest_normal * fi.eps / 2


def close(got, want, tol, t, what):
    """got within tol of want, and a rounding to t more; want nan: not compared."""
    g = f64(got)
    tol = tol * (1 + torch.finfo(TYPES[t]).eps) + stored(want, t)
    ok = np.isnan(want) | (np.abs(g - want) <= tol)
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} outside, worst {np.nanmax(np.where(ok, 0, np.abs(g - want) / np.maximum(tol, 1e-300)))}"


def guards_hold(buf, view_cols, shift, what):
    b = buf.detach().float().cpu()
    g = 0xA5 if buf.dtype == torch.uint8 else GUARD
    assert (b[..., :shift] == g).all() and (b[..., shift + view_cols:] == g).all(), what


def offsets_of(groups, M):
    return None if groups is None else torch.tensor(groups, dtype=torch.int32, device=DEV)


def run_forward(M, N, K, t, ty, act, bias, res, keep, groups, pad=0, shift=0, seed=0):
    r = np.random.default_rng(seed)
    G = 1 if groups is None else len(groups) - 1
    x = normal(r, M, K, t=t)
    w = normal(r, G, N, K, t=t, scale=1 / np.sqrt(max(K, 1)))
    b = normal(r, G, N, t="f32", scale=0.3) if bias else None
    res_t = normal(r, M, N, t=ty) if res else None
    dx, dw = strided(x, pad, shift)[1], strided(w, pad, shift)[1]
    db = None if b is None else b.to(DEV)
    dr = None if res_t is None else strided(res_t, pad, shift)[1]
    ybuf, y = strided(torch.full((M, N), GUARD, dtype=TYPES[ty]), pad, shift)
    z = zs = None
    if keep == "z16":
        zbuf, z = strided(torch.full((M, N), GUARD, dtype=TYPES[t]), pad, shift)
    elif keep == "mx8":
        zbuf, zc = strided(torch.full((M, N), 0xA5, dtype=torch.uint8), pad, shift)
        z = zc, strided(torch.full((M, -(-N // 32)), 0xA5, dtype=torch.uint8), pad, shift)[1]
    off = offsets_of(groups, M)
    if G == 1 and groups is None:
        dw, db = dw[0], None if db is None else db[0]
    assert ll.linear16_nt(dx, dw, db, ACT[act], dr, y, Z=z, offsets=off) is y
    torch.cuda.synchronize()
    spans = ref.bounds(groups, M)
    zr, size = ref.linear(f64(x), f64(w), None if b is None else f64(b), spans)
    tz = (K + 1) * STEP * size
    want = ref.act(zr, act) + (f64(res_t) if res else 0)
    tol = 1.13 * tz + 16 * H32 * (1 + np.abs(zr)) + (H32 * (np.abs(want) + 1e-30) if res else 0)
    close(y, want, tol, ty, "y")
    guards_hold(ybuf, N, shift, "y's guards")
    outside = np.isnan(zr[:, 0]) if N else np.zeros(M, bool)
    assert (f64(y)[outside] == GUARD).all()
    if keep == "z16":
        close(z, zr, tz, t, "z")
        guards_hold(zbuf, N, shift, "z's guards")
        assert (f64(z)[outside] == GUARD).all()
    elif keep == "mx8":
        codes, scales = z[0].cpu().numpy(), z[1].cpu().numpy()
        guards_hold(zbuf, N, shift, "codes' guards")
        assert (codes[outside] == 0xA5).all() and (scales[outside] == 0xA5).all()
        got = ref.mx8_values(codes, scales)
        for c in range(0, N, 32):
            zb, tb = zr[:, c:c + 32], tz[:, c:c + 32]
            top = (np.abs(zb) + tb).max(axis=1, keepdims=True)
            tol8 = 2.0 ** -4 * (np.abs(zb) + tb) + 2.0 ** -10 * 2 * top / 448 + tb
            ok = np.isnan(zb) | (np.abs(got[:, c:c + 32] - zb) <= tol8)
            assert ok.all(), f"z in 8 bits: {(~ok).sum()} outside at column {c}"
    return y


SHAPES = [(1, 1, 1), (1, 7, 3), (2, 64, 64), (3, 65, 33), (17, 128, 72), (64, 100, 8), (65, 257, 136), (129, 130, 200),
          (130, 300, 65), (33, 1000, 512)]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_shapes(shape, t):
    M, N, K = shape
    run_forward(M, N, K, t, t, "silu", True, False, "", None, seed=M + N + K)
    run_forward(M, N, K, t, "f32", "none", False, True, "mx8", None, seed=M + N + K + 1)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("keep", ["", "z16", "mx8"])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_forward_writeback(act, keep, ty):
    run_forward(150, 200, 128, "bf16", ty, act, True, True, keep, None, seed=3)


GROUPS = [[0, 5, 5, 130, 131, 200], [3, 70, 199], [0, 0, 0, 200], [200, 200], [0] * 70 + [9, 130, 200], [0, 1, 2, 3, 4],
          [7, 3, 90, 50, 400], [-5, 60, 2 ** 31 - 1]]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("groups", GROUPS)
def test_forward_groups(groups, t):
    """Empty groups, rows of no group, more groups than a wave has lanes, and offsets that
    descend or lie outside the rows."""
    run_forward(200, 136, 72, t, t, "gelu", True, True, "mx8", groups, seed=len(groups))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (8, 8), (3, 5)])
def test_forward_strides(pad, shift, t):
    run_forward(140, 152, 136, t, t, "relu", True, True, "z16", None, pad, shift, seed=9)
    run_forward(140, 152, 136, t, "f32", "gelu_tanh", True, True, "mx8", [0, 40, 133], pad, shift, seed=10)


@pytest.mark.parametrize("shape", [(4100, 3900, 72), (4096, 4096, 128)])
def test_forward_large_tiles(shape):
    run_forward(*shape, "bf16", "bf16", "silu", True, False, "mx8", None, seed=21)


def test_forward_large_tiles_by_group():
    run_forward(4100, 4000, 64, "f16", "f32", "none", False, True, "", [0, 1000, 1000, 1257, 4000], seed=22)


def test_forward_without_inner_dimension():
    b = torch.randn(40, device=DEV)
    y = torch.full((5, 40), GUARD, dtype=torch.bfloat16, device=DEV)
    x, w = torch.empty((5, 0), dtype=torch.bfloat16, device=DEV), torch.empty((40, 0), dtype=torch.bfloat16, device=DEV)
    ll.linear16_nt(x, w, b, ll.ACT_RELU, None, y)
    assert torch.equal(y, b.clamp(min=0).bfloat16().expand(5, 40))


def test_residual_in_place():
    r = np.random.default_rng(2)
    x, w = normal(r, 130, 64, t="bf16").to(DEV), normal(r, 96, 64, t="bf16", scale=0.1).to(DEV)
    for t in (torch.bfloat16, torch.float32):
        res = torch.randn((130, 96), device=DEV).to(t)
        y = torch.empty_like(res)
        ll.linear16_nt(x, w, None, ll.ACT_SILU, res, y)
        ll.linear16_nt(x, w, None, ll.ACT_SILU, res, res)
        assert torch.equal(y, res)


def test_infinities_and_nan():
    """They stay in their rows; a block of 8 bits that has one is NaN as a whole."""
    x = torch.randn((40, 64), device=DEV).bfloat16()
    w = torch.randn((96, 64), device=DEV).bfloat16()
    x[3, 5], x[20, 1], w[50] = float("nan"), float("inf"), 0
    y, y0 = (torch.empty((40, 96), device=DEV) for _ in range(2))
    q = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(40, 96))
    ll.linear16_nt(x, w, None, ll.ACT_NONE, None, y, Z=q)
    clean = x.clone()
    clean[3, 5] = clean[20, 1] = 0
    ll.linear16_nt(clean, w, None, ll.ACT_NONE, None, y0)
    rows = [i for i in range(40) if i not in (3, 20)]
    assert torch.equal(y[rows], y0[rows]) and y[3].isnan().all() and not y[20].isfinite().any()
    assert (q[1][3] == 255).all() and (q[1][20] == 255).all() and (q[0][3] == 0).all() and (q[1][rows] < 255).all()
    ll.linear16_nt(x, w, None, ll.ACT_RELU, None, y)
    assert (y[3] == 0).all() and not torch.signbit(y[3]).any()


# ---- 8 bits -----------------------------------------------------------------

@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 33), (5, 64), (7, 100), (4, 1000), (65, 257)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_quantise_to_the_bit(shape, t, pad, shift):
    r = np.random.default_rng(shape[1])
    x = normal(r, *shape, t=t) * (10.0 ** torch.as_tensor(r.integers(-3, 3, shape))).to(TYPES[t])
    x[0, 0] = 0
    if shape[1] > 64:
        x[0, 32:64] = 0
        x[-1, 40] = float("inf")
        x[-1, 3] = float("nan")
    want = ref.mx8_quantize(f64(x))
    cbuf, codes = strided(torch.zeros(shape, dtype=torch.uint8), pad, shift)
    sbuf, scales = strided(torch.zeros((shape[0], -(-shape[1] // 32)), dtype=torch.uint8), pad, shift)
    ll.mx8_quantize(strided(x, pad, shift)[1], codes, scales)
    assert (scales.cpu().numpy() == want[1]).all() and (codes.cpu().numpy() == want[0]).all()
    guards_hold(cbuf, shape[1], shift, "codes")
    guards_hold(sbuf, scales.shape[1], shift, "scales")
    ybuf, y = strided(torch.zeros(shape, dtype=TYPES[t]), pad, shift)
    ll.mx8_dequantize(codes, scales, y)
    v = ref.mx8_values(*want)
    with np.errstate(over="ignore"):
        v = torch.as_tensor(v).to(TYPES[t]).double().numpy()   # (float64 to 16 bits rounds once)
    assert np.array_equal(f64(y), v, equal_nan=True)
    guards_hold(ybuf, shape[1], shift, "values")


def test_quantise_scales_of_all_sizes():
    """A block's largest over the whole range of FP32, next to each border of its scale."""
    e = np.arange(-149, 128)
    tops = np.concatenate([np.float32(2.0) ** e] + [np.float32(m) * np.float32(2.0) ** np.clip(e, -120, 126)
                                                    for m in (1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.1)])
    r = np.random.default_rng(1)
    x = (tops[:, None] * np.concatenate([np.ones((tops.size, 1)), r.uniform(-1, 1, (tops.size, 31))], axis=1)).astype(np.float32)
    want = ref.mx8_quantize(x)
    codes, scales = (torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(*x.shape))
    ll.mx8_quantize(torch.as_tensor(x).to(DEV), codes, scales)
    assert (scales.cpu().numpy() == want[1]).all()
    assert (codes.cpu().numpy() == want[0]).all()
    y = torch.empty(x.shape, device=DEV)
    ll.mx8_dequantize(codes, scales, y)
    assert np.array_equal(f64(y), ref.mx8_values(*want).astype(np.float32).astype(np.float64))


def test_dequantise_every_code():
    """Every code under every scale: FP32 and bfloat16 as float64 rounds to them."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8)
    v = ref.mx8_values(codes.cpu().numpy(), scales.cpu().numpy())
    for t in ("f32", "bf16", "f16"):
        y = torch.empty((256, 256), dtype=TYPES[t], device=DEV)
        ll.mx8_dequantize(codes, scales, y)
        # (values have four bits: a rounding to FP32 on the way to 16 bits changes nothing)
        want = torch.as_tensor(v).float().to(TYPES[t])
        same = (y.cpu() == want) | (y.cpu().isnan() & want.isnan())
        assert same.all(), (t, (~same).nonzero()[:5], (~same).sum())


# ---- gradients ----------------------------------------------------------------

def run_grad_act(M, N, t, ty, act, keep, bias, groups, pad=0, shift=0, seed=0, dz=True):
    r = np.random.default_rng(seed)
    G = 1 if groups is None else len(groups) - 1
    dy, z = normal(r, M, N, t=ty), normal(r, M, N, t=t, scale=2.0)
    zr, zd = f64(z), strided(z, pad, shift)[1]
    if keep == "mx8":
        codes, scales = ref.mx8_quantize(zr)
        zr = ref.mx8_values(codes, scales)
        zd = strided(codes, pad, shift)[1], strided(scales, pad, shift)[1]
    if act == "none":
        zd = None
    buf, out = strided(torch.full((M, N), GUARD, dtype=TYPES[t]), pad, shift)
    db = torch.full((G, N) if groups else (N,), GUARD, device=DEV) if bias else None
    dyd = strided(dy, pad, shift)[1]
    if dz:
        assert ll.linear16_grad_act(dyd, zd, ACT[act], out, db, offsets=offsets_of(groups, M)) is out
    spans = ref.bounds(groups, M)
    want = f64(dy) * ref.slope(zr, act)
    size = np.abs(f64(dy)) * (1 + np.abs(zr))   # each slope is a few operations on at most |z| and 1
    inside = np.zeros(M, bool)
    for a, e in spans:
        inside[a:e] = True
    close(out, np.where(inside[:, None], want, np.nan), 24 * H32 * size, t, "dz")
    assert (f64(out)[~inside] == GUARD).all()
    guards_hold(buf, N, shift, "dz's guards")
    if bias:
        wb = np.stack([want[a:e].sum(0) for a, e in spans])
        tb = np.stack([(M * H32 * np.abs(want[a:e]) + 24 * H32 * size[a:e]).sum(0) for a, e in spans])
        close(db.reshape(G, N), wb, tb, "f32", "dbias")


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("keep", ["z16", "mx8"])
def test_grad_act(t, act, keep):
    run_grad_act(77, 200, t, t, act, keep, True, None, seed=1)
    run_grad_act(77, 200, t, "f32", act, keep, True, [0, 5, 5, 60, 70], seed=2)
    run_grad_act(77, 203, t, t, act, keep, False, None, 3, 1, seed=3)


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (15, 64), (16, 65), (17, 500), (300, 512), (40, 513), (5, 3001)])
def test_grad_act_shapes(shape):
    run_grad_act(*shape, "bf16", "bf16", "silu", "mx8", True, None, seed=4)
    run_grad_act(*shape, "f16", "f32", "gelu", "z16", True, None, 1, 1, seed=5)


@pytest.mark.parametrize("groups", GROUPS)
def test_grad_act_groups(groups):
    run_grad_act(200, 72, "bf16", "bf16", "gelu_tanh", "mx8", True, groups, seed=6)


def test_grad_act_many_rows():
    """Chunks of 64 rows, and more of them than the joining workgroup has shares."""
    run_grad_act(4500, 1000, "bf16", "bf16", "silu", "z16", True, [0, 100, 4400], seed=7)
    run_grad_act(4500, 1000, "bf16", "f32", "none", "z16", True, None, seed=8)


def test_grad_act_in_place_and_without_rows():
    dy, z = (torch.randn((33, 70), device=DEV).bfloat16() for _ in range(2))
    out = torch.empty_like(dy)
    ll.linear16_grad_act(dy, z, ll.ACT_SILU, out)
    a, b = dy.clone(), z.clone()
    ll.linear16_grad_act(a, z, ll.ACT_SILU, a)
    ll.linear16_grad_act(dy, b, ll.ACT_SILU, b)
    assert torch.equal(a, out) and torch.equal(b, out)
    db = torch.full((3, 70), GUARD, device=DEV)
    e = torch.empty((0, 70), dtype=torch.bfloat16, device=DEV)
    ll.linear16_grad_act(e, e.clone(), ll.ACT_SILU, e.clone(), db, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert (db == 0).all()


def test_grad_act_of_extreme_values():
    """Slopes go to 0 and 1; no infinity meets a zero. NaN stays."""
    z = torch.tensor([[-float("inf"), -3e38, -1e20, -200.0, 200.0, 1e20, 3e38, float("inf"), float("nan")]], device=DEV).bfloat16()
    dy = torch.ones_like(z)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        out = ll.linear16_grad_act(dy, z, ACT[act], torch.empty_like(z)).float().cpu()[0]
        assert out[:4].abs().max() == 0 and (out[4:8] == 1).all(), (act, out)
        assert out[8].isnan() or act == "relu"
        w = torch.ones((1, 1), device=DEV).bfloat16()
        y = torch.empty((9, 1), device=DEV)
        ll.linear16_nt(z.t().contiguous(), w, None, ACT[act], None, y)
        y = y.cpu()[:, 0]
        assert (y[:4] == 0).all() and (y[4:8] == z.float().cpu()[0, 4:8]).all(), (act, y)


def run_grad_input(M, N, K, t, tx, groups, pad=0, shift=0, seed=0):
    r = np.random.default_rng(seed)
    G = 1 if groups is None else len(groups) - 1
    dz, w = normal(r, M, N, t=t), normal(r, G, N, K, t=t, scale=1 / np.sqrt(max(N, 1)))
    buf, out = strided(torch.full((M, K), GUARD, dtype=TYPES[tx]), pad, shift)
    wd = strided(w, pad, shift)[1]
    ll.linear16_grad_input(strided(dz, pad, shift)[1], wd if groups else wd[0], out, offsets=offsets_of(groups, M))
    want, size = ref.grad_input(f64(dz), f64(w), ref.bounds(groups, M))
    close(out, want, N * STEP * size, tx, "dx")
    assert (f64(out)[np.isnan(want)] == GUARD).all()
    guards_hold(buf, K, shift, "dx's guards")


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_grad_input(shape, t):
    run_grad_input(*shape, t, t, None, seed=1)
    run_grad_input(*shape, t, "f32", None, 8, 0, seed=2)


@pytest.mark.parametrize("groups", GROUPS)
def test_grad_input_groups(groups):
    run_grad_input(200, 72, 136, "bf16", "bf16", groups, seed=3)
    run_grad_input(200, 70, 135, "f16", "f32", groups, 1, 3, seed=4)


def test_grad_input_large_tiles():
    run_grad_input(4100, 72, 3904, "bf16", "bf16", None, seed=5)
    run_grad_input(4100, 64, 4000, "f16", "f32", [0, 1000, 1000, 1257, 4000], seed=6)


def run_grad_weight(M, N, K, t, tw, beta, keep, groups, pad=0, shift=0, seed=0):
    r = np.random.default_rng(seed)
    G = 1 if groups is None else len(groups) - 1
    dz, x = normal(r, M, N, t=t), normal(r, M, K, t=t)
    xr, xd = f64(x), strided(x, pad, shift)[1]
    if keep == "mx8":
        codes, scales = ref.mx8_quantize(xr)
        xr = ref.mx8_values(codes, scales)
        xd = strided(codes, pad, shift)[1], strided(scales, pad, shift)[1]
    dw0 = normal(r, G, N, K, t=tw) if beta else torch.full((G, N, K), float("nan"), dtype=TYPES[tw])
    buf, out = strided(dw0, pad, shift)
    ll.linear16_grad_weight(strided(dz, pad, shift)[1], xd, out if groups else out[0], beta=beta, offsets=offsets_of(groups, M))
    want, size = ref.grad_weight(f64(dz), xr, ref.bounds(groups, M))
    if beta:
        want = want + beta * f64(dw0)
        size = size + np.abs(beta * f64(dw0))
    close(out, want, (M + 2) * STEP * size, tw, "dw")
    guards_hold(buf, K, shift, "dw's guards")


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("keep", ["", "mx8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_grad_weight(shape, keep, t):
    M, N, K = shape
    run_grad_weight(M, N, K, t, t, 0.0, keep, None, seed=1)
    run_grad_weight(M, N, K, t, "f32", 0.5, keep, None, 8, 0, seed=2)


@pytest.mark.parametrize("keep", ["", "mx8"])
@pytest.mark.parametrize("groups", GROUPS)
def test_grad_weight_groups(groups, keep):
    run_grad_weight(200, 72, 136, "bf16", "bf16", 0.0, keep, groups, seed=3)
    run_grad_weight(200, 70, 135, "f16", "f32", 1.0, keep, groups, 1, 3, seed=4)


@pytest.mark.parametrize("keep", ["", "mx8"])
def test_grad_weight_large_tiles(keep):
    run_grad_weight(72, 4100 - 4, 3904, "bf16", "f32", 1.0, keep, None, seed=5)
    run_grad_weight(333, 1160, 2048, "f16", "f16", 0.0, keep, [0, 100, 100, 257, 300], seed=6)


def test_grad_weight_of_large_binary16_values():
    """65504 becomes 65536 in 8 bits, which binary16 does not hold: it enters the product as
    65504."""
    x = torch.full((4, 40), 65504.0, device=DEV).half()
    q = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(4, 40))
    ll.mx8_quantize(x, *q)
    dz = torch.zeros((4, 16), device=DEV).half()
    dz[1] = 1
    dw = ll.linear16_grad_weight(dz, q, torch.empty((16, 40), device=DEV))
    assert (dw == 65504).all()


def test_equal_calls_give_equal_bits():
    r = np.random.default_rng(0)
    x, w = normal(r, 300, 640, t="bf16").to(DEV), normal(r, 500, 640, t="bf16").to(DEV)
    dz = normal(r, 300, 500, t="bf16").to(DEV)
    first = None
    for _ in range(3):
        y, dx, dw = (torch.empty(s, device=DEV) for s in ((300, 500), (300, 640), (500, 640)))
        db = torch.empty(500, device=DEV)
        ll.linear16_nt(x, w, None, ll.ACT_SILU, None, y)
        ll.linear16_grad_act(dz, dz, ll.ACT_SILU, torch.empty_like(dz), db)
        ll.linear16_grad_input(dz, w, dx)
        ll.linear16_grad_weight(dz, x, dw)
        got = (y, dx, dw, db)
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
