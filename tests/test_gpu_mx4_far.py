"""The 4-bit operators at the far end of the sizes: launches that have to be cut into
several. Inputs repeat a short pattern, whose outcome the plain float64 implementation
gives; the whole output is compared with it."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import quantize, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def equal_to_pattern(got, pattern):
    """Whether row k of `got` is row k % len(pattern) of `pattern`, for all rows."""
    n, p = got.shape[0], pattern.shape[0]
    whole = n // p * p
    return torch.equal(got[:whole].view(n // p, p, -1), pattern.expand(n // p, *pattern.shape)) and \
        torch.equal(got[whole:], pattern[:n - whole])


@pytest.mark.parametrize("M,K", [(2, 2 ** 29 + 1000), (33, 2 ** 27 + 77)])
def test_quantize_columns_past_a_launch(M, K):
    """More columns than one launch has work items for."""
    period = 1009
    x = torch.as_tensor(np.random.default_rng(1).standard_normal((M, period)) * np.exp2(np.arange(period) % 13 - 6)).half()
    X = x.to(DEV).repeat(1, K // period + 1)[:, :K]
    (_, nq), (_, ns) = ll.mx4_shapes(K, M)
    codes, scales = (torch.full((K, n), 0xAB, dtype=torch.uint8, device=DEV) for n in (nq, ns))
    ll.mx4_quantize(X, codes, scales, trans=True)
    want_c, want_s = quantize(x.double().numpy().T)
    assert equal_to_pattern(scales, torch.as_tensor(want_s).to(DEV))
    assert equal_to_pattern(codes, torch.as_tensor(want_c).to(DEV))


def repeated(v, rows):
    """v's rows over and over, on the GPU."""
    v = torch.as_tensor(v).to(DEV)
    return v.repeat(rows // v.shape[0] + 1, 1)[:rows]


def integers(r, which, rows, K):
    """A operand of whole numbers (packed values are multiples of 1 up to 12): arguments
    of its pattern, float64 values. Sums stay below 2^24, so results are exact."""
    if which == "16":
        x = torch.as_tensor(r.integers(-8, 9, (rows, K)))
        return (x.to(torch.bfloat16),), x.double().numpy()
    (_, nq), (_, ns) = ll.mx4_shapes(rows, K)
    c, s = r.integers(0, 256, (rows, nq), np.uint8), np.full((rows, ns), 128, np.uint8)
    return (c, s), values(c, s, K)


PERIOD = 1009
# more tiles (of 16 rows, by kernel of 4 or 8 waves) or rows than a launch has work items for
MANY_ROWS = [(2 ** 28 + 33, 4, 4, "tiny"), (2 ** 27 + 70, 3, 300, "stream_")]
MANY_COLUMNS = [(3, 2 ** 28 + 33, 20, "tiny"), (1, 2 ** 27 + 70, 512, "rows"), (2, 2 ** 27 + 70, 300, "stream_")]


def product(a, b, C, K):
    if len(a) == 2:
        ll.gemm_mx4f32_nt(*a, *b, C, K=K)
    else:
        ll.gemm_bf16mx4f32_nt(*a, *b, C)


@pytest.mark.parametrize("which", ["mx4", "16"])
@pytest.mark.parametrize("M,N,K,kernel", MANY_ROWS)
def test_rows_past_a_launch(M, N, K, kernel, which):
    assert ll.mx4_chosen_kernel(M, N, K, ll.A_MX4 if which == "mx4" else ll.A_BF16).startswith(kernel)
    r = np.random.default_rng(2)
    (a, av), (b, bv) = integers(r, which, PERIOD, K), integers(r, "mx4", N, K)
    C = torch.full((M, N), float("nan"), device=DEV)
    product([repeated(v, M) for v in a], [torch.as_tensor(v).to(DEV) for v in b], C, K)
    assert np.abs(av).max() * 12 * K < 2 ** 24
    assert equal_to_pattern(C, torch.as_tensor(av @ bv.T).float().to(DEV))


@pytest.mark.parametrize("which", ["mx4", "16"])
@pytest.mark.parametrize("M,N,K,kernel", MANY_COLUMNS)
def test_columns_past_a_launch(M, N, K, kernel, which):
    assert ll.mx4_chosen_kernel(M, N, K, ll.A_MX4 if which == "mx4" else ll.A_BF16).startswith(kernel)
    r = np.random.default_rng(3)
    (a, av), (b, bv) = integers(r, which, M, K), integers(r, "mx4", PERIOD, K)
    C = torch.full((M, N), float("nan"), device=DEV)
    product([torch.as_tensor(v).to(DEV) for v in a], [repeated(v, N) for v in b], C, K)
    want = torch.as_tensor(av @ bv.T).float().to(DEV)
    for m in range(M):
        assert equal_to_pattern(C[m][:, None], want[m][:, None])
