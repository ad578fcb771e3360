"""The products' promise that every decoded value of a 4-bit operand enters exactly,
whatever its scale, at the largest scale bytes: under 253 and 254 (2^126 and 2^127) a
value reaches 6 * 2^127, past the largest bfloat16 and FP32. The other operand is small
or zero, so that the products and their sums are ordinary FP32 numbers.

Tolerance as in test_gpu_mx4: (K + 8) half-steps of FP32 (2^-24) of the sum of the
terms' magnitudes, and 2^-126 a term."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF_STEP = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def operands(which, M, N, K, seed, all_far, pad):
    r = np.random.default_rng(seed)
    (_, nq), (_, ns) = ll.mx4_shapes(N, K)
    codes = r.integers(0, 256, (N, nq), np.uint8)
    scales = r.integers(250, 255, (N, ns)).astype(np.uint8)
    if not all_far:   # a few such blocks among ordinary ones, in the first row and the last
        scales = r.integers(115, 136, (N, ns)).astype(np.uint8)
        scales[0, 0], scales[N // 2, ns // 2], scales[N - 1, ns - 1] = 253, 254, 254
    if which == "mx4":
        (_, nq), (_, ns) = ll.mx4_shapes(M, K)
        ca, sa = r.integers(0, 256, (M, nq), np.uint8), r.integers(85, 96, (M, ns)).astype(np.uint8)
        ca[M // 2] = 0
        av, a = values(ca, sa, K), [place(ca, pad), place(sa, pad)]
    else:
        x = torch.as_tensor(r.standard_normal((M, K)) * 2.0 ** (-18 if which == "f16" else -40)).to(TYPES[which])
        x[torch.as_tensor(r.random((M, K)) < 0.1)] = 0
        x[M // 2] = 0
        av, a = x.double().numpy(), [place(x, pad)]
    return a, av, codes, scales


def place(v, pad):
    v = torch.as_tensor(v)
    out = torch.zeros((v.shape[0], v.shape[1] + pad), dtype=v.dtype, device=DEV)[:, :v.shape[1]]
    return out.copy_(v)


def product(which, a, codes, scales, C, K, alpha=1.0, beta=0.0):
    if which == "mx4":
        return ll.gemm_mx4f32_nt(*a, codes, scales, C, alpha, beta, K=K)
    return (ll.gemm_f16mx4f32_nt if which == "f16" else ll.gemm_bf16mx4f32_nt)(*a, codes, scales, C, alpha, beta)


# one row (a wave to a row of B, two, none), few rows, shares of K, short and tiny K,
# tiles of 128 and 256 with rows on and off 16 bytes, with a rest of K
SIZES = [(1, 40, 6184), (1, 5, 9000), (1, 30, 100), (5, 33, 1000), (33, 300, 11008), (64, 64, 512), (70, 90, 31),
         (1300, 1700, 32), (1501, 1603, 201), (300, 520, 1056), (512, 768, 1024), (2100, 2200, 544)]


@pytest.mark.parametrize("which", ["mx4", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("all_far,pad", [(True, 0), (False, 0), (False, 1)])
def test_product_under_the_largest_scales(M, N, K, all_far, pad, which):
    a, av, codes, scales = operands(which, M, N, K, 1, all_far, pad)
    bv = values(codes, scales, K)
    C = torch.full((M, N), float("nan"), device=DEV)
    product(which, a, place(codes, pad), place(scales, pad), C, K)
    got, want, size = C.double().cpu().numpy(), av @ bv.T, np.abs(av) @ np.abs(bv).T
    assert np.abs(want).max() < 2.0 ** 127 and size.max() < 2.0 ** 127
    bad = ~(np.abs(got - want) <= (K + 8) * (HALF_STEP * size + 2.0 ** -126))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, {np.isnan(got).sum()} NaN, {np.isinf(got).sum()} infinite"
    assert (got[M // 2] == 0).all()


@pytest.mark.parametrize("which", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 6184), (5, 33, 1000), (512, 768, 1024), (700, 520, 1056)])
def test_not_finite_beside_the_largest_scales(M, N, K, which):
    """NaN blocks and an infinity of A stay what they are where a row of B has such a
    scale too; other rows and columns stay finite; alpha and beta enter once."""
    a, av, codes, scales = operands(which, M, N, K, 2, False, 0)
    scales[3, 1] = 255
    a[0][0, 40] = float("inf")
    av[0, 40] = np.inf
    c0 = np.random.default_rng(3).standard_normal((M, N)).astype(np.float32)
    C = torch.as_tensor(c0).to(DEV)
    product(which, a, place(codes, 0), place(scales, 0), C, K, 1.5, 0.5)
    got = C.double().cpu().numpy()
    assert np.isnan(got[:, 3]).all()
    code = codes[:, 20] & 7
    others = np.arange(N) != 3
    assert (np.isnan(got[0]) == (code == 0))[others].all() and not np.isfinite(got[0]).any()
    if M > 1:
        with np.errstate(invalid="ignore"):
            bv = values(codes, scales, K)[others]
            want, size = 1.5 * (av[1:] @ bv.T) + 0.5 * c0[1:, others], 1.5 * (np.abs(av[1:]) @ np.abs(bv).T) + 0.5 * np.abs(c0[1:, others])
        assert (np.abs(got[1:, others] - want) <= (K + 8) * (HALF_STEP * size + 2.0 ** -126)).all()


@pytest.mark.parametrize("which", ["mx4", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 6184), (1, 30, 100), (5, 33, 1000), (33, 300, 11008), (70, 90, 31), (1300, 1700, 128),
                                   (1000, 1500, 1577), (2100, 2200, 1600)])
def test_quantised_nan_reaches_the_product(M, N, K, which):
    """A block that held a NaN or an infinity has codes of 0 under the NaN scale: its row
    is NaN in the product all the same, and no other, also against zeros of A."""
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    w = torch.randn((N, K), generator=g, device=DEV)
    w[3, K // 2], w[N - 1, K - 1] = float("nan"), float("-inf")

    def pack(t):
        (c, s) = ll.mx4_shapes(*t.shape)
        return ll.mx4_quantize(t, *(torch.empty(v, dtype=torch.uint8, device=DEV) for v in (c, s)))

    x = torch.randn((M, K), generator=g, device=DEV)
    x[M // 2] = 0
    a = pack(x) if which == "mx4" else (x.to(TYPES[which]),)
    C = torch.zeros((M, N), device=DEV)
    product(which, a, *pack(w), C, K)
    want = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    want[:, [3, N - 1]] = True
    assert torch.equal(torch.isnan(C), want) and bool(torch.isfinite(C[~want]).all())
