"""The 16-bit layer at its edges: codes whose rows end inside a word, GELU to FP32. References in float64 on
the device by torch. Tolerances as in test_gpu_linear16: a sum of n products is off by at most
n steps of 2^-23 of the sum of their magnitudes, and stored with half a step of its type."""
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
