"""The tile kernels of the products with a 4-bit operand, each case checked to take the
kernel it is meant for: 256 x 256 tiles with direct copies (whole ones, last rounds in
halves, a half past the last row), 128 x 128 with copies and through registers, panels
of scales that follow one another, what K leaves past whole stages, tiles moved back
at the edges, alpha and beta, far and NaN scales in the first, a middle and the last
panel and past them.

Tolerance as in test_gpu_mx4: (K + 8) half-steps of FP32 (2^-24) of the sum of the
terms' magnitudes, and 2^-126 a term. What FP32 cannot hold has to be infinite."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF_STEP = 2.0 ** -24
WHICH = {"mx4": ll.A_MX4, "f16": ll.A_F16, "bf16": ll.A_BF16}


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def place(v, aligned):
    """A device copy with rows on 16 bytes, 16 bytes or more apart from one another, or
    with odd ones; bytes between them are 0xAB."""
    v = torch.as_tensor(v)
    per = 16 // v.element_size()
    ld = (v.shape[1] // per + 2) * per + (0 if aligned else 1)
    buf = torch.empty((v.shape[0], ld), dtype=v.dtype, device=DEV)
    buf.view(torch.uint8).fill_(0xAB)
    out = buf[:, :v.shape[1]]
    out.copy_(v)
    return out


def packed(r, rows, K, lo=115, hi=135):
    (_, nq), (_, ns) = ll.mx4_shapes(rows, K)
    return r.integers(0, 256, (rows, nq), np.uint8), r.integers(lo, hi + 1, (rows, ns)).astype(np.uint8)


class Case:
    def __init__(self, which, M, N, K, aligned, kernel, seed):
        cus = torch.cuda.get_device_properties(0).multi_processor_count
        assert ll.mx4_chosen_kernel(M, N, K, WHICH[which], aligned, True, cus) == kernel
        r = np.random.default_rng(seed)
        self.which, self.M, self.N, self.K, self.aligned = which, M, N, K, aligned
        self.codes, self.scales = packed(r, N, K)
        if which == "mx4":
            self.a, self.sa = packed(r, M, K, 119, 139)
        else:
            x = torch.as_tensor(r.standard_normal((M, K)) * np.exp2(r.integers(-3, 4, (1, K))))
            self.a = x.to(torch.float16 if which == "f16" else torch.bfloat16)
        self.c0 = torch.as_tensor(r.standard_normal((M, N)).astype(np.float32))

    def run(self, alpha, beta):
        C = place(self.c0 if beta else torch.full((self.M, self.N), float("nan")), self.aligned)
        guard = C.as_strided((self.M, C.stride(0)), (C.stride(0), 1))
        keep = guard.clone()
        b = place(self.codes, self.aligned), place(self.scales, self.aligned)
        if self.which == "mx4":
            ll.gemm_mx4f32_nt(place(self.a, self.aligned), place(self.sa, self.aligned), *b, C, alpha, beta, K=self.K)
        else:
            f = ll.gemm_f16mx4f32_nt if self.which == "f16" else ll.gemm_bf16mx4f32_nt
            f(place(self.a, self.aligned), *b, C, alpha, beta)
        assert torch.equal(guard[:, self.N:].contiguous().view(torch.int32), keep[:, self.N:].contiguous().view(torch.int32))
        return C

    def exact(self, alpha, beta):
        a = torch.as_tensor(values(self.a, self.sa, self.K)).to(DEV) if self.which == "mx4" else self.a.to(DEV).double()
        b = torch.as_tensor(values(self.codes, self.scales, self.K)).to(DEV)
        c = self.c0.to(DEV).double()
        return (alpha * (a @ b.t().contiguous()) + (beta * c if beta else 0),
                abs(alpha) * (a.abs() @ b.abs().t().contiguous()) + (abs(beta) * c.abs() if beta else 0))

    def check(self, alpha=1.0, beta=0.0):
        got, (want, size) = self.run(alpha, beta).double(), self.exact(alpha, beta)
        bad = ~((got - want).abs() <= (self.K + 8) * (HALF_STEP * size + 2.0 ** -126))
        top = float(torch.finfo(torch.float32).max)
        bad &= size <= top            # (a partial sum may pass what FP32 holds; NaN is compared below)
        bad |= (want.abs() > top) & ~torch.isinf(got)
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"
        assert torch.equal(torch.isnan(got), torch.isnan(want))


BIG, SMALL = "tile_256x256", "tile_128x128"
# whole tiles and a last round in halves, one of which lies past the last row; a last
# round of whole tiles; all tiles in halves
LARGE = [(2100, 9000, 1577), (5000, 3000, 1568), (2100, 2200, 1600)]


@pytest.mark.parametrize("which", list(WHICH))
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (-1.5, 0.5)])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_tiles(M, N, K, alpha, beta, which):
    Case(which, M, N, K, True, BIG, 1).check(alpha, beta)


@pytest.mark.parametrize("which", list(WHICH))
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (-1.5, 0.5)])
@pytest.mark.parametrize("M,N,K", [(1000, 1500, 1577), (1024, 1536, 2048)])
def test_small_tiles(M, N, K, alpha, beta, aligned, which):
    Case(which, M, N, K, aligned, SMALL, 2).check(alpha, beta)


PLACES = [(2100, 9000, 1577, True, BIG), (1000, 1500, 1577, True, SMALL), (1000, 1500, 1577, False, SMALL)]


@pytest.mark.parametrize("which", list(WHICH))
@pytest.mark.parametrize("M,N,K,aligned,kernel", PLACES)
def test_far_scales_in_some_blocks(M, N, K, aligned, kernel, which):
    """Scales past binary16 (and past bfloat16: the two largest) in single blocks of a few
    rows: the first panel, a middle one, the last, and the block that K ends in."""
    c = Case(which, M, N, K, aligned, kernel, 3)
    last = c.scales.shape[1] - 1
    places = [(0, 0, 90), (N // 2, last // 2, 145), (N - 1, last, 60), (N - 70, last - 3, 160), (17, 16, 250)]
    if which != "mx4":
        c.a *= 2.0 ** -8
        places += [(130, 1, 253), (N - 2, last, 254)]
    for n, b, s in places:
        c.scales[n, b] = s
    c.check(1.0, 0.5)


@pytest.mark.parametrize("which", list(WHICH))
@pytest.mark.parametrize("M,N,K,aligned,kernel", PLACES)
def test_nan_scales(M, N, K, aligned, kernel, which):
    """A NaN block makes its column of C NaN (of A in 4 bits, its row), and nothing else."""
    c = Case(which, M, N, K, aligned, kernel, 4)
    last = c.scales.shape[1] - 1
    for n, b in ((0, 0), (127, 20), (N // 2, 33), (N - 1, last)):
        c.scales[n, b] = 255
    if which == "mx4":
        for m, b in ((1, last), (130, 0), (M - 1, 17)):
            c.sa[m, b] = 255
    else:
        c.a[M - 2, 40] = float("nan")
    c.check()


@pytest.mark.parametrize("which", list(WHICH))
@pytest.mark.parametrize("M,N,K,aligned,kernel", PLACES)
def test_tiles_repeat_bit_for_bit(M, N, K, aligned, kernel, which):
    c = Case(which, M, N, K, aligned, kernel, 5)
    first = c.run(1.0, 0.0).clone()
    for _ in range(2):
        assert torch.equal(c.run(1.0, 0.0), first)
