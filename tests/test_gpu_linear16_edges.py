"""The 16-bit layer at its edges: codes whose rows end inside a word, codes by kernel, NaN blocks,
GELU to FP32, kept 8 bits against the call's own sums, the gradients of many groups, few rows in
shares, the bias's gradient alone. References in float64 on the device by torch. Tolerances as in
test_gpu_linear16: a sum of n products is off by at most n steps of 2^-23 of the sum of their
magnitudes, and stored with half a step of its type."""
import math

import pytest

import linear16_reference as ref
import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STEP = 2.0 ** -23


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def randn(seed, *shape, t="bf16", scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPES[t])


def close(got, want, size, n, what):
    tol = n * STEP * size
    if got.dtype != torch.float32:
        fi = torch.finfo(got.dtype)
        tol = tol * (1 + fi.eps) + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps / 2
    ok = (got.double() - want).abs() <= tol
    assert ok.all(), f"{what}: {(~ok).sum().item()} of {ok.numel()} outside, first at {(~ok).nonzero()[0].tolist()}"


def both(a, b):
    """a^T b and the sums of its terms' magnitudes."""
    return a.double().t().contiguous() @ b.double(), a.double().abs().t().contiguous() @ b.double().abs()


def offsets_of(groups):
    return None if groups is None else torch.tensor(groups, dtype=torch.int32, device=DEV)


def in_8_bits(x, ld):
    """x's codes in rows ld apart with NaN codes between them, and its scales; and their values."""
    M, K = x.shape
    codes = torch.full((M, ld), 0x7F, dtype=torch.uint8, device=DEV)[:, :K]
    scales = torch.empty(ll.mx8_shapes(M, K)[1], dtype=torch.uint8, device=DEV)
    ll.mx8_quantize(x, codes, scales)
    return (codes, scales), ll.mx8_dequantize(codes, scales, torch.empty((M, K), device=DEV))


def weight_kernel(dz, q, groups):
    """The kernel that linear16_grad_weight takes for these operands, by their alignment too."""
    (M, N), K = dz.shape, q[0].shape[1]
    aligned = (dz.data_ptr() % 16 == 0 and dz.stride(0) % 8 == 0 and N % 8 == 0
               and q[0].data_ptr() % 16 == 0 and q[0].stride(0) % 16 == 0)
    return ll.linear16_chosen_kernel(ll.L16_GRAD_WEIGHT, M, N, K, 1 if groups is None else len(groups) - 1, aligned)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(200, 264, 1001, 1008, None, "small"), (200, 264, 1002, 1008, None, "small"),
                                   (333, 72, 1003, 1008, [0, 70, 70, 300], "small"), (65, 8, 1, 16, None, "small"),
                                   (1032, 6400, 2001, 2016, None, "large"), (1032, 6400, 2002, 2016, None, "large"),
                                   (1025, 4096, 2303, 2304, [0, 300, 300, 1025], "large")], ids=str)
def test_weight_gradient_from_codes_that_end_inside_a_word(shape, t):
    """Codes on 16 bytes whose rows are no whole words: the last columns take part in every row."""
    M, N, K, ld, groups, kernel = shape
    dz, x = randn(1, M, N, t=t), randn(2, M, K, t=t)
    q, xr = in_8_bits(x, ld)
    assert weight_kernel(dz, q, groups) == kernel
    spans = ref.bounds(groups, M)
    dw = torch.empty((len(spans), N, K), device=DEV)
    ll.linear16_grad_weight(dz, q, dw if groups else dw[0], offsets=offsets_of(groups))
    for g, (a, e) in enumerate(spans):
        close(dw[g], *both(dz[a:e], xr[a:e]), M, "dw")


H32 = 2.0 ** -24


def gelu_grid():
    """Normal values, and all of [-12, 12]; and where the normal ones end."""
    z = torch.cat([randn(7, 50000, t="f32"), torch.linspace(-12, 12, 48001, device=DEV), torch.zeros(7, device=DEV)])
    return z, 50000


def parts(z):
    """The normal distribution function, and its density times |z|, in 64 bits."""
    return 0.5 * torch.erfc(-z / math.sqrt(2)), z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("M", [1, 130])
def test_gelu_to_fp32(M):
    """Z is the bias alone. From -1 on: the function is 1/2 + z P or 1 - h, six half-steps with the product; on
    the negative side h's operations are ten of its own and its exponent's three at z^2 / 2 each.
    In the norm two roundings of at most half a step, evenly spread: 0.82 half-steps."""
    z, normal = gelu_grid()
    y = torch.empty((M, z.numel()), device=DEV)
    zeros = torch.zeros((max(M, z.numel()), 8), device=DEV).bfloat16()
    ll.linear16_nt(zeros[:M], zeros[:z.numel()], z, ll.ACT_GELU, None, y)
    zd = z.double()
    want = zd * parts(zd)[0]
    tol = H32 * want.abs() * torch.where(zd >= -1, 6.0, 10 + 2 * zd * zd)
    off = (y.double() - want).abs()
    assert (off <= tol).all(), (off / tol).nan_to_num().max()
    rms = (off[:, :normal].norm() / want[:normal].expand(M, -1).norm()).item()
    assert rms <= H32, rms


@pytest.mark.parametrize("ty", ["f16", "f32"])
def test_gelu_slope_to_fp32(ty):
    """The bias's gradient of one row is its slope. The function as above, the density's part six half-steps and its
    exponent's, and their sum."""
    z = gelu_grid()[0].half()[None]
    dy = torch.ones_like(z).to(TYPES[ty])
    db = torch.empty(z.shape[1], device=DEV)
    dz = ll.linear16_grad_act(dy, z, ll.ACT_GELU, torch.empty_like(z), db)
    zd = z[0].double()
    c, d = parts(zd)
    want = c + torch.where(zd < 0, -d, d)
    tol = H32 * torch.where(zd >= -1, 6 * c + (6 + 2 * zd * zd) * d, (10 + 2 * zd * zd) * (c + d))
    off = (db.double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert ((dz[0].double() - want).abs() <= tol + 2.0 ** -11 * want.abs() + 2.0 ** -25).all()


def test_kept_8_bits_are_the_formats_of_the_calls_own_sums():
    """Z in 8 bits is to the bit what mx8_quantize makes of the same call's FP32 sums, and a call repeats itself:
    what another order of sums gives differs from it only where a sum lies next to a border between codes."""
    M, N, K = 2047, 11008, 4096
    assert ll.linear16_chosen_kernel(ll.L16_FORWARD, M, N, K) == "large"
    x, w, b = randn(1, M, K), randn(2, N, K, scale=K ** -0.5), randn(3, N, t="f32", scale=0.2)
    z = torch.empty((M, N), device=DEV)
    ll.linear16_nt(x, w, b, ll.ACT_NONE, None, z)
    want = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
    ll.mx8_quantize(z, *want)
    first = None
    for i in range(5):
        y = torch.full((M, N), float("nan"), device=DEV).bfloat16()
        q = tuple(torch.full(s, 0x7F - i, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
        ll.linear16_nt(x, w, b, ll.ACT_GELU, None, y, Z=q)
        assert torch.equal(q[0], want[0]) and torch.equal(q[1], want[1])
        assert first is None or torch.equal(y, first)
        first = y
    # (the order of sums of the library's FP32 product)
    other = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
    zo = torch.matmul(x.float(), w.float().t()) + b
    ll.mx8_quantize(zo, *other)
    va, vb = (ll.mx8_dequantize(*q, torch.empty((M, N), device=DEV)).double() for q in (want, other))
    differ = va != vb
    size = (x.double().abs() @ w.double().abs().t() + b.double().abs())[differ]
    exact = (x.double() @ w.double().t() + b.double())[differ]
    border = ((va + vb) / 2)[differ]
    assert ((exact - border).abs() <= (K + 1) * STEP * size).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(512, 304, 272, 272, None, "small"), (300, 136, 208, 208, [0, 3, 250, 300], "small"),
                                   (1000, 136, 200, 208, [5, 5, 390, 999], "small"), (512, 304, 264, 264, None, "small_any"),
                                   (300, 136, 200, 200, [0, 3, 250, 300], "small_any"), (500, 135, 256, 256, None, "small_any"),
                                   (1032, 6400, 2000, 2000, None, "large")], ids=str)
def test_weight_gradient_from_codes_by_kernel(shape, t):
    """Each kernel over many stages, named by the operands' own alignment; a block that is NaN makes its columns of its
    group NaN and no others, any code under the scale byte 255 among them."""
    M, N, K, ld, groups, kernel = shape
    dz, x = randn(1, M, N, t=t), randn(2, M, K, t=t)
    q, xr = in_8_bits(x, ld)
    assert weight_kernel(dz, q, groups) == kernel
    spans = ref.bounds(groups, M)
    before = randn(3, len(spans), N, K, t="f32")
    dw = before.clone()

    def call(q):
        ll.linear16_grad_weight(dz, q, dw if groups else dw[0], beta=1.0, offsets=offsets_of(groups))

    call(q)
    clean = dw.clone()
    for g, (a, e) in enumerate(spans):
        want, size = both(dz[a:e], xr[a:e])
        close(dw[g], want + before[g].double(), size + before[g].double().abs(), e - a + 1, "dw")
    a = spans[-1][0] + 7                      # a row of the last group, its blocks 1 and the last
    q[1][a, 1] = q[1][a, -1] = 255
    dw.copy_(before)
    call(q)
    nan = torch.zeros(K, dtype=torch.bool, device=DEV)
    nan[32:64] = nan[(K - 1) // 32 * 32:] = True
    assert dw[-1][:, nan].isnan().all() and torch.equal(dw[-1][:, ~nan], clean[-1][:, ~nan])
    assert torch.equal(dw[:-1], clean[:-1])


@pytest.mark.parametrize("M", [900, 7000])
def test_gradients_of_many_groups(M):
    """Five thousand groups, most of them empty or of a row."""
    G, N, K = 5000, 40, 64
    r = torch.Generator().manual_seed(M)
    off = torch.cat([torch.tensor([0, M - 3]), torch.randint(0, M - 3, (G - 1,), generator=r)]).sort().values.to(torch.int32).to(DEV)
    group = torch.searchsorted(off[1:].long(), torch.arange(M - 3, device=DEV), right=True)
    dz, x, w = randn(1, M, N), randn(2, M, K), randn(3, G, N, K)
    for op in (ll.L16_GRAD_INPUT, ll.L16_GRAD_WEIGHT):
        assert ll.linear16_chosen_kernel(op, M, N, K, G) == "small"
    dx = torch.full((M, K), 7.0, device=DEV)
    ll.linear16_grad_input(dz, w, dx, offsets=off)
    d = dz[:-3].double()[:, None]
    close(dx[:-3], torch.matmul(d, w[group].double())[:, 0], torch.matmul(d.abs(), w[group].double().abs())[:, 0], N, "dx")
    assert (dx[-3:] == 7).all()
    outer = dz[:-3].double()[:, :, None] * x[:-3].double()[:, None, :]
    want, size = (torch.zeros((G, N, K), dtype=torch.float64, device=DEV).index_add_(0, group, v) for v in (outer, outer.abs()))
    most = int(torch.bincount(group).max())
    dw = torch.full((G, N, K), float("nan"), device=DEV)
    ll.linear16_grad_weight(dz, x, dw, offsets=off)
    close(dw, want, size, most, "dw")
    db, out = torch.full((G, N), float("nan"), device=DEV), torch.full((M, N), 7.0, device=DEV).bfloat16()
    ll.linear16_grad_act(dz, x[:, :N].contiguous(), ll.ACT_RELU, out, db, offsets=off)
    slope = (x[:-3, :N] > 0).double()
    v = dz[:-3].double() * slope
    assert torch.equal(out[:-3].double(), v) and (out[-3:] == 7).all()
    want, size = (torch.zeros((G, N), dtype=torch.float64, device=DEV).index_add_(0, group, u) for u in (v, v.abs()))
    close(db, want, size, most, "dbias")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("align", [16, 4, 2])
@pytest.mark.parametrize("case", [(1, 200, 4097, None), (33, 130, 8200, None), (64, 72, 4104, None), (2, 64, 8192, [0, 1, 2]),
                                  (70, 200, 8200, [3, 20, 20, 61]), (120, 64, 4104, [0, 64, 120])], ids=str)
def test_few_rows_in_shares(case, align, t):
    """Few rows a group, the inner dimension in shares, with all of the write-back; rows on 16, 4 and 2 bytes."""
    M, N, K, groups = case
    if align == 16:
        K = K // 8 * 8
    G = 1 if groups is None else len(groups) - 1
    assert ll.linear16_chosen_kernel(ll.L16_FORWARD, M, N, K, G, align == 16) == ("rows" if align == 16 else "rows_any")
    need = ll.linear16_workspace_size(ll.L16_FORWARD, M, N, K, G)
    assert need >= 2 * 4 * M * N
    # rows that begin and lie 16, 4 and 2 bytes apart, NaN around them
    shift, ld = {16: (0, K + 8), 4: (2, (K + 5) // 4 * 4 + 2), 2: (1, K + 2 + K % 2 + 1)}[align]

    def laid(a):
        v = torch.full((*a.shape[:-1], ld), float("nan"), dtype=a.dtype, device=DEV)[..., shift:shift + K]
        v.copy_(a)
        return v

    x, w = laid(randn(1, M, K, t=t)), laid(randn(2, G, N, K, t=t, scale=K ** -0.5))
    for v in (x, w):
        assert (v.data_ptr() | 2 * v.stride(-2)) % 16 % (2 * align) == align % 16
    b, r = randn(3, G, N, t="f32"), randn(4, M, N, t=t)
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    y = torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV)
    q = tuple(torch.full(s, 0xA5, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
    off = offsets_of(groups)
    ll.linear16_nt(x, w if groups else w[0], b if groups else b[0], ll.ACT_RELU, r, y, Z=q, offsets=off, workspace=ws)
    y2 = torch.full_like(y, 7.0)
    ll.linear16_nt(x, w if groups else w[0], b if groups else b[0], ll.ACT_RELU, r, y2, offsets=off)
    assert torch.equal(y, y2)
    outside = torch.ones(M, dtype=torch.bool, device=DEV)
    values = ll.mx8_dequantize(*q, torch.empty((M, N), device=DEV)).double()
    for g, (a, e) in enumerate(ref.bounds(groups, M)):
        outside[a:e] = False
        if a == e:
            continue
        z, size = both(x[a:e].t(), w[g].t())
        z, size = z + b[g].double(), size + b[g].double().abs()
        want = z.clamp(min=0) + r[a:e].double()
        close(y[a:e], want, size + want.abs(), K + 2, "y")
        err = (K + 1) * STEP * size
        top = torch.nn.functional.pad(z.abs() + err, (0, -N % 32)).view(e - a, -1, 32).amax(2).repeat_interleave(32, 1)[:, :N]
        assert ((values[a:e] - z).abs() <= 2.0 ** -4 * (z.abs() + err) + 2.0 ** -9 * top / 448 + err).all()
    assert (y[outside] == 7).all() and (q[0][outside] == 0xA5).all() and (q[1][outside] == 0xA5).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("groups", [None, [2, 30, 30, 97]])
@pytest.mark.parametrize("eight", [False, True])
def test_bias_gradient_alone(act, groups, eight):
    """The C call without DZ: the sums are to the bit those of the call that writes it."""
    M, N = 100, 203
    dy, z = randn(1, M, N), randn(2, M, N)
    G = 1 if groups is None else len(groups) - 1
    off = offsets_of(groups)
    held, zq = z, (None, None)
    if eight:
        held = zq = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
        ll.mx8_quantize(z, *zq)
    kind = getattr(ll, "ACT_" + act.upper())
    want = torch.empty((G, N) if groups else (N,), device=DEV)
    ll.linear16_grad_act(dy, held, kind, torch.empty_like(dy), want, offsets=off)
    got = torch.full_like(want, float("nan"))
    ws = torch.empty(ll.linear16_grad_act_workspace_size(M, N, G), dtype=torch.uint8, device=DEV)

    def at(v):
        return None if v is None else v.data_ptr()

    status = ll.load().linear16_grad_act(M, N, ll.TYPE_BF16, kind, ll.TYPE_BF16, at(dy), N, G, at(off), None if eight else at(z), N,
                                         at(zq[0]), N, at(zq[1]), (N + 31) // 32, None, N, at(got), at(ws), ws.numel(),
                                         torch.cuda.current_stream().cuda_stream)
    assert status == ll.OK
    assert torch.equal(got, want)


def test_an_activation_past_a_c_int():
    """Refused, not cut to its lower 32 bits."""
    x, w = randn(1, 4, 32), randn(2, 8, 32)
    y = torch.full((4, 8), 7.0, device=DEV).bfloat16()
    for act in (2 ** 32, 2 ** 32 + 1, -2 ** 32 + 4, 2 ** 40):
        with pytest.raises(ValueError):
            ll.linear16_nt(x, w, None, act, None, y)
        with pytest.raises(ValueError):
            ll.linear16_grad_act(y, y, act, y)
    assert (y == 7).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [40, 300])
def test_empty_axes_by_group(M, t):
    """Sums of nothing are zeros (and the bias, or beta's part) in the rows of groups, and rows outside stay."""
    N, K, groups = 72, 40, [3, 20, 20, M - 5]
    off = offsets_of(groups)
    b = randn(3, 3, N, t="f32")
    y = torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV)
    q = tuple(torch.full(s, 0xA5, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
    none = torch.empty((M, 0), dtype=TYPES[t], device=DEV)
    ll.linear16_nt(none, torch.empty((3, N, 0), dtype=TYPES[t], device=DEV), b, ll.ACT_RELU, None, y, Z=q, offsets=off)
    z = ll.mx8_dequantize(*q, torch.empty((M, N), device=DEV))
    for g, (a, e) in enumerate(ref.bounds(groups, M)):
        row = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(1, N))
        ll.mx8_quantize(b[g:g + 1], *row)
        assert torch.equal(y[a:e], b[g].clamp(min=0).to(TYPES[t]).expand(e - a, N))
        assert torch.equal(z[a:e], ll.mx8_dequantize(*row, torch.empty((1, N), device=DEV)).expand(e - a, N))
    dx = torch.full((M, K), 7.0, dtype=TYPES[t], device=DEV)
    ll.linear16_grad_input(none, torch.empty((3, 0, K), dtype=TYPES[t], device=DEV), dx, offsets=off)
    outside = torch.ones(M, dtype=torch.bool, device=DEV)
    outside[3:M - 5] = False
    assert (dx[~outside] == 0).all()
    for v in (y, dx):
        assert (v[outside] == 7).all()
    assert (q[0][outside] == 0xA5).all() and (q[1][outside] == 0xA5).all()
    for beta in (0.0, 0.5):
        dw = torch.full((3, N, K), 3.0, device=DEV)
        ll.linear16_grad_weight(torch.empty((0, N), dtype=TYPES[t], device=DEV), torch.empty((0, K), dtype=TYPES[t], device=DEV), dw,
                                beta=beta, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
        assert (dw == 3 * beta).all()
