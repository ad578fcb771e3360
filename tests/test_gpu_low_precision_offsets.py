"""The 4-bit operators and the residual norms with rows so far apart that offsets pass
2^31 elements and 2^32 bytes, against the same calls on rows side by side (whose
correctness the other tests hold), bit for bit; and tensors that take several launches,
whose rows repeat a pattern and have to have its results.

A product's kernel goes by the alignment of its rows, which is the same on both sides."""
import numpy as np
import pytest

import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U8, F32, BF = torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def far(t, ld):
    """t with its rows ld elements apart."""
    buf = torch.empty(((t.shape[0] - 1) * ld + t.shape[1],), dtype=t.dtype, device=DEV)
    v = buf.as_strided(tuple(t.shape), (ld, 1))
    v.copy_(t)
    return v


def near(t, odd):
    """t with rows on 16 bytes, or with odd ones."""
    per = 16 // t.element_size()
    return far(t.to(DEV), (t.shape[1] // per + 1) * per + odd)


def packed(r, rows, K):
    (_, nq), (_, ns) = ll.mx4_shapes(rows, K)
    return [torch.as_tensor(r.integers(0, 256, (rows, nq), np.uint8)), torch.as_tensor(r.integers(118, 132, (rows, ns)).astype(np.uint8))]


def product(a, b, C, K):
    if len(a) == 2:
        ll.gemm_mx4f32_nt(*a, *b, C, 1.5, 0.5, K=K)
    else:
        ll.gemm_bf16mx4f32_nt(*a, *b, C, 1.5, 0.5)


# (the last one: rows 2^24 bytes apart or more take no direct copies)
PRODUCTS = [(1, 300, 4096, 2 ** 24, "rows"), (40, 70, 320, 2 ** 27, "stream_"), (1300, 1700, 20, 2 ** 22, "tiny"),
            (1300, 1700, 128, 2 ** 22, "short"), (1000, 1500, 1577, 2 ** 22, "tile_128x128"),
            (2100, 2200, 1600, 2 ** 21, "tile_256x256")]


@pytest.mark.parametrize("which", ["mx4", "16"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("M,N,K,step,kernel", PRODUCTS)
def test_products(M, N, K, step, kernel, odd, which):
    form = ll.A_MX4 if which == "mx4" else ll.A_BF16
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    if odd and kernel == "tile_256x256":
        kernel = "tile_128x128"
    assert ll.mx4_chosen_kernel(M, N, K, form, not odd, True, cus).startswith(kernel)
    r = np.random.default_rng(1)
    a = packed(r, M, K) if which == "mx4" else [torch.as_tensor(r.standard_normal((M, K))).to(BF)]
    b, c = packed(r, N, K), torch.as_tensor(r.standard_normal((M, N)).astype(np.float32))
    want, got = near(c, odd), far(c.to(DEV), step + odd)
    product([near(t, odd) for t in a], [near(t, odd) for t in b], want, K)
    product([far(t.to(DEV), step + odd) for t in a], [far(t.to(DEV), step + odd) for t in b], got, K)
    assert torch.equal(got, want)


def test_rows_too_far_for_copies():
    """Rows on 16 bytes but 2^24 or more apart: the plan without copies."""
    M, N, K, ld = 300, 400, 2048, 2 ** 24
    r = np.random.default_rng(2)
    a, b = packed(r, M, K), packed(r, N, K)
    want, got = torch.zeros((M, N), device=DEV), torch.zeros((M, N), device=DEV)
    ll.gemm_mx4f32_nt(*(near(t, 1) for t in a), *(near(t, 1) for t in b), want, K=K)
    ll.gemm_mx4f32_nt(*(far(t.to(DEV), ld) for t in a), *(far(t.to(DEV), ld) for t in b), got, K=K)
    assert torch.equal(got, want)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_quantisation(dtype, trans):
    M, K, ld = 301, 333, 2 ** 23 + 1
    x = torch.as_tensor(np.random.default_rng(3).standard_normal((M, K))).to(dtype).to(DEV)
    rows, n = (K, M) if trans else (M, K)
    new = lambda k: torch.zeros(ll.mx4_shapes(rows, n)[k], dtype=U8, device=DEV)  # noqa: E731
    c, s = ll.mx4_quantize(x, new(0), new(1), trans=trans)
    fc, fs = ll.mx4_quantize(far(x, ld), far(new(0), ld), far(new(1), ld), trans=trans)
    assert torch.equal(fc, c) and torch.equal(fs, s)
    y = torch.zeros((rows, n), dtype=dtype, device=DEV)
    assert torch.equal(ll.mx4_dequantize(fc, fs, far(y, ld)), ll.mx4_dequantize(c, s, y))


@pytest.mark.parametrize("N", [100, 1500, 5000, 9000])
def test_norms(N):
    M, ld = 300, 2 ** 23 + 8
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    new = lambda t: torch.randn((M, N), generator=g, device=DEV).to(t)  # noqa: E731
    y, x, dxo, dh, w = new(F32), new(BF), new(BF), new(BF), torch.rand((N,), generator=g, device=DEV)
    ws = torch.empty((ll.rmsnorm_grad_workspace_size(M, N),), dtype=U8, device=DEV)
    outs = []
    for place in (lambda t: t.clone(), lambda t: far(t, ld)):
        out = [place(torch.zeros((M, N), dtype=t, device=DEV)) for t in (BF, BF, F32, BF)]
        vec = [torch.zeros((N,), device=DEV) for _ in range(3)]
        ll.rmsnorm_residual(place(y), w, w, 0.7, place(x), w, out[0], out[1])
        ll.rmsnorm_residual_grad(place(dxo), place(dh), place(y), w, w, 0.7, place(x), w, out[2], out[3], *vec, ws)
        outs.append(out + vec)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ---- several launches -------------------------------------------------------------

def pattern(rows, cols, dtype, period=1009):
    """(pattern, it over and over for `rows` rows)."""
    p = torch.as_tensor(np.random.default_rng(5).standard_normal((period, cols))).to(dtype).to(DEV)
    return p, p.repeat(rows // period + 1, 1)[:rows]


def follows(got, want):
    n, p = got.shape[0], want.shape[0]
    whole = n // p * p
    step = (1 << 30) // (p * got.shape[1]) * p + p
    for m in range(0, whole, step):
        part = got[m:min(m + step, whole)]
        if not torch.equal(part.view(-1, p, got.shape[1]), want.expand(part.shape[0] // p, *want.shape)):
            return False
    return torch.equal(got[whole:], want[:n - whole])


def test_quantisation_of_more_values_than_a_launch_takes():
    M, K = 2 ** 28 + 999, 32      # 2^30 groups of 8 values to a launch
    p, x = pattern(M, K, BF)
    new = lambda rows, k: torch.zeros(ll.mx4_shapes(rows, K)[k], dtype=U8, device=DEV)  # noqa: E731
    want = ll.mx4_quantize(p, new(1009, 0), new(1009, 1))
    got = ll.mx4_quantize(x, new(M, 0), new(M, 1))
    assert follows(got[0], want[0]) and follows(got[1], want[1])
    y = ll.mx4_dequantize(*got, x)
    assert follows(y, ll.mx4_dequantize(*want, torch.empty_like(p)))


def test_long_rows_past_a_launch_or_a_grid():
    """Rows longer than a workgroup's registers: the forward's walk past 2^20 rows, and
    the gradient's first launch of 2^20 rows."""
    M = (1 << 20) + 1015
    p, x = pattern(M, 16400, BF)
    want, h = torch.empty_like(p), torch.empty_like(x)
    ll.rmsnorm_residual(None, None, None, 1.0, p, None, None, want)
    ll.rmsnorm_residual(None, None, None, 1.0, x, None, None, h)
    assert follows(h, want)
    del h, x, p
    torch.cuda.empty_cache()
    N = 8200
    p, x = pattern(M, N, BF)
    small = torch.empty((ll.rmsnorm_grad_workspace_size(1009, N),), dtype=U8, device=DEV)
    large = torch.empty((ll.rmsnorm_grad_workspace_size(M, N),), dtype=U8, device=DEV)
    want, dx = torch.empty_like(p), torch.empty_like(x)
    ll.rmsnorm_residual_grad(p, p, None, None, None, 1.0, p, None, None, want, None, None, None, small)
    ll.rmsnorm_residual_grad(x, x, None, None, None, 1.0, x, None, None, dx, None, None, None, large)
    assert follows(dx, want)


@pytest.mark.parametrize("which", ["mx4", "f16", "bf16"])
@pytest.mark.parametrize("K", [257, 320, 384, 511])
def test_inner_dimensions_between_one_wave_and_the_tiles(K, which):
    """K past the one-wave kernel's and short of the tiles' under a large output, exact on
    whole numbers below 2^24."""
    from mx4_reference import values
    M, N = 1303, 1701
    r = np.random.default_rng(6)
    b = packed(r, N, K)
    b[1].fill_(128)
    if which == "mx4":
        a = packed(r, M, K)
        a[1].fill_(128)
        av = values(a[0].numpy(), a[1].numpy(), K)
    else:
        x = torch.as_tensor(r.integers(-8, 9, (M, K)))
        a, av = [x.to(torch.float16 if which == "f16" else BF)], x.double().numpy()
    C = torch.full((M, N), float("nan"), device=DEV)
    args = [t.to(DEV) for t in a + b]
    if which == "mx4":
        ll.gemm_mx4f32_nt(*args, C, K=K)
    else:
        (ll.gemm_f16mx4f32_nt if which == "f16" else ll.gemm_bf16mx4f32_nt)(*args, C)
    assert np.array_equal(C.double().cpu().numpy(), av @ values(b[0].numpy(), b[1].numpy(), K).T)
