"""The 16-bit layer at its edges: codes whose rows end inside a word. References in float64 on
the device by torch. Tolerances as in test_gpu_linear16: a sum of n products is off by at most
n steps of 2^-23 of the sum of their magnitudes, and stored with half a step of its type."""
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
