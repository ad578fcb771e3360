"""The microscaled 4-bit format on the GPU: quantisation along rows and columns,
the way back, and the products with one or both operands in it, against a
plain float64 implementation (mx4_reference), at odd sizes, strides and
alignments, extreme scales, infinities and NaN.

Tolerances. Quantisation and its inverse have one right answer each (the
inverse rounds once to the output type, which numpy and torch do alike), so
they are compared for equality. A product's inputs enter exactly; its FP32 sum
of K terms, in whatever order, is off by at most (K + 8) half-steps of FP32
(2^-24) of the sum of the terms' magnitudes, and alpha, beta and the final
additions by a few half-steps more of what they act on; below FP32's smallest
normal value, 2^-126, each term may be lost whole. Integer-valued inputs
whose sums stay below 2^24 units give the exact result."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import quantize, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = 2.0 ** -24


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def rng(seed):
    return np.random.default_rng(seed)


def strided(a, pad=0, shift=0, fill=0xAB):
    """A device copy of a 2-D array, rows `pad` elements apart, base `shift` in."""
    a = torch.as_tensor(a)
    buf = torch.empty((a.shape[0], shift + a.shape[1] + pad), dtype=a.dtype, device=DEV)
    buf.view(torch.uint8).fill_(fill)
    v = buf[:, shift:shift + a.shape[1]]
    v.copy_(a)
    return buf, v


def empty_packed(rows, K, pad=0, shift=0):
    (r, c), (_, s) = ll.mx4_shapes(rows, K)
    return strided(np.zeros((r, c), np.uint8), pad, shift), strided(np.zeros((r, s), np.uint8), pad, shift)


def spread(r, rows, cols):
    """Values whose blocks differ in size, with zeros, ties and whole blocks of 0."""
    x = r.standard_normal((rows, cols)) * np.exp2(r.integers(-12, 12, (rows, cols // 32 + 1)).repeat(32, axis=1)[:, :cols])
    x[r.random((rows, cols)) < 0.05] = 0
    ties = r.random((rows, cols)) < 0.2
    x[ties] = r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], ties.sum()) * r.choice([-1, 1], ties.sum())
    if cols > 64:
        x[::3, 32:64] = 0
    return x


SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (1, 4096), (7, 255), (33, 257), (257, 97), (300, 1001), (64, 2048)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1), (16, 0)])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize(M, K, kind, pad, shift, trans):
    x = torch.as_tensor(spread(rng(M * 1000 + K), M, K)).to(TYPES[kind])
    want_c, want_s = quantize(x.double().numpy().T if trans else x.double().numpy())
    rows, n = (K, M) if trans else (M, K)
    (cb, c), (sb, s) = empty_packed(rows, n, pad, shift)
    cb0, sb0 = cb.clone(), sb.clone()
    ll.mx4_quantize(strided(x, pad, shift)[1], c, s, trans=trans)
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(c.cpu().numpy(), want_c)
    # nothing outside the codes and scales is written
    c.zero_(), s.zero_()
    assert torch.equal(cb, cb0) and torch.equal(sb, sb0)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_extremes(kind, trans):
    """Infinities, NaN, subnormals, the largest values: one kind to a block."""
    t = TYPES[kind]
    fi = torch.finfo(t)
    specials = [0.0, float("inf"), -float("inf"), float("nan"), fi.max, -fi.max, fi.tiny, fi.smallest_normal / 8,
                fi.smallest_normal * 7, fi.tiny * 0.9, 1.0, 6.5, 7.999]
    x = torch.as_tensor(spread(rng(5), 13 * 4, 32 * 4)).to(t)
    for i, v in enumerate(specials):
        for j in range(4):
            if j < 3:
                x[4 * i + j, 32 * j:32 * j + 32] *= 0.0 if abs(v) < 1e-3 else 1.0
            x[4 * i + j, 32 * j + 5 + i] = v
    want_c, want_s = quantize(x.double().numpy().T if trans else x.double().numpy())
    (_, c), (_, s) = empty_packed(*(x.shape[::-1] if trans else x.shape))
    ll.mx4_quantize(x.to(DEV), c, s, trans=trans)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(c.cpu().numpy(), want_c)


@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", SHAPES + [(256, 64)])
def test_dequantize(M, K, kind, pad, shift):
    """Every code under every scale byte (256 x 64 walks all 256 of them)."""
    r = rng(M + K)
    (cs, ss) = ll.mx4_shapes(M, K)
    codes, scales = r.integers(0, 256, cs, np.uint8), r.integers(0, 256, ss, np.uint8)
    if (M, K) == (256, 64):
        scales[:, 0] = np.arange(256)
    with np.errstate(over="ignore"):
        want = torch.as_tensor(values(codes, scales, K)).to(TYPES[kind])
    yb, y = strided(torch.zeros((M, K), dtype=TYPES[kind]), pad, shift)
    keep = yb.clone()
    ll.mx4_dequantize(strided(codes, pad, shift)[1], strided(scales, pad, shift)[1], y)
    got = y.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    y.zero_()
    assert torch.equal(yb.view(torch.uint8), keep.view(torch.uint8))


# ---- products -------------------------------------------------------------------

def packed_case(r, rows, K, lo=115, hi=135):
    cs, ss = ll.mx4_shapes(rows, K)
    return r.integers(0, 256, cs, np.uint8), r.integers(lo, hi + 1, ss, np.uint8)


def a_operand(which, r, M, K, pad, shift, lo=115, hi=135):
    """(arguments of A, its float64 values)."""
    if which == "mx4":
        c, s = packed_case(r, M, K, 254 - hi, 254 - lo)   # B's scales mirrored: products near 1
        return (strided(c, pad, shift)[1], strided(s, pad, shift)[1]), values(c, s, K)
    t = TYPES[which]
    x = torch.as_tensor(r.standard_normal((M, K)) * np.exp2(r.integers(-3, 4, (1, K)))).to(t)
    return (strided(x, pad, shift)[1],), x.double().numpy()


def product(which, args, B, SB, C, alpha, beta, K):
    if which == "mx4":
        ll.gemm_mx4f32_nt(*args, B, SB, C, alpha, beta, K=K)
    else:
        (ll.gemm_f16mx4f32_nt if which == "f16" else ll.gemm_bf16mx4f32_nt)(*args, B, SB, C, alpha, beta)


def check(which, M, N, K, alpha=1.0, beta=0.0, pad=0, shift=0, lo=115, hi=135, seed=1):
    r = rng(seed)
    args, av = a_operand(which, r, M, K, pad, shift)
    c, s = packed_case(r, N, K, lo, hi)
    bv = values(c, s, K)
    c0 = r.standard_normal((M, N)).astype(np.float32)
    cb, C = strided(c0 if beta else np.full((M, N), np.nan, np.float32), pad, shift)
    keep = cb.clone()
    product(which, args, strided(c, pad, shift)[1], strided(s, pad, shift)[1], C, alpha, beta, K)
    got = C.double().cpu().numpy()
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    want, size = alpha * want, abs(alpha) * size
    if beta:
        want, size = want + beta * c0, size + abs(beta) * np.abs(c0)
    bad = ~(np.abs(got - want) <= (K + 8) * (HALF_STEP * size + 2.0 ** -126))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside the bound, worst {np.nanmax(np.abs(got - want) / size)}"
    C.zero_()
    keep[:, shift:shift + N] = 0
    assert torch.equal(cb.view(torch.uint8), keep.view(torch.uint8))


WHICH = ["mx4", "f16", "bf16"]
SIZES = [(1, 1, 1), (1, 16, 32), (2, 3, 31), (3, 17, 33), (16, 16, 128), (17, 100, 257), (1, 300, 4096), (5, 33, 1000),
         (64, 64, 512), (65, 130, 384), (33, 96, 11008), (255, 257, 320), (256, 256, 1024), (300, 520, 96), (257, 300, 777),
         (512, 512, 544), (1000, 700, 64), (130, 1030, 2080), (600, 640, 4128)]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, which):
    check(which, M, N, K)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("alpha,beta", [(1.5, 0.5), (-0.5, 1.0), (0.0, 0.25), (2.0, -1.0)])
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (20, 70, 100), (300, 300, 512), (512, 768, 1024)])
def test_product_alpha_beta(M, N, K, alpha, beta, which):
    check(which, M, N, K, alpha, beta, seed=2)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (5, 3), (16, 0), (16, 16)])
@pytest.mark.parametrize("M,N,K", [(3, 50, 200), (70, 90, 320), (260, 520, 512)])
def test_product_strides(M, N, K, pad, shift, which):
    """Row strides and bases off 16 bytes, and on them with padding between rows."""
    check(which, M, N, K, 1.0, 0.5, pad, shift, seed=3)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", [(2, 40, 160), (70, 70, 256), (300, 300, 512)])
@pytest.mark.parametrize("lo,hi", [(0, 30), (60, 104), (103, 105), (139, 142), (150, 190)])
def test_product_scales(M, N, K, lo, hi, which):
    """Scales far from 1, those past binary16's own range among them."""
    check(which, M, N, K, lo=lo, hi=hi, seed=4)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", [(1, 70, 96), (40, 70, 416), (300, 512, 1056)])
def test_product_exact_on_integers(M, N, K, which):
    r = rng(7)
    c, s = packed_case(r, N, K, 128, 128)      # multiples of 1 up to 12
    if which == "mx4":
        ca, sa = packed_case(r, M, K, 128, 128)
        args, av = (torch.as_tensor(ca).to(DEV), torch.as_tensor(sa).to(DEV)), values(ca, sa, K)
    else:
        x = torch.as_tensor(r.integers(-8, 9, (M, K))).to(TYPES[which])
        args, av = (x.to(DEV),), x.double().numpy()
    C = torch.full((M, N), float("nan"), device=DEV)
    product(which, args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
    want = av @ values(c, s, K).T
    assert np.abs(av).max() * 12 * K < 2 ** 24
    assert np.array_equal(C.double().cpu().numpy(), want)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", [(2, 40, 160), (70, 90, 256), (300, 300, 512)])
def test_product_nan_and_infinity_stay_in_their_rows(M, N, K, which):
    """A scale of 255 makes its block NaN: the rows (columns) of C that read it,
    and no others, are NaN. An infinity of A makes its row infinite or NaN."""
    r = rng(8)
    c, s = packed_case(r, N, K)
    s[N // 2, (K // 32) // 2] = 255
    args, av = a_operand(which, r, M, K, 0, 0)
    if which == "mx4":
        args[1][M // 2, 1] = 255
    else:
        args[0][M // 2, 40] = float("inf")
        args[0][0, 3] = float("nan")
    C = torch.zeros((M, N), device=DEV)
    product(which, args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
    bad = ~torch.isfinite(C).cpu()
    want = torch.zeros((M, N), dtype=torch.bool)
    want[:, N // 2] = True
    want[M // 2, :] = True
    if which != "mx4":
        want[0, :] = True
        # against a code of 0 an infinity gives NaN, else an infinity of the code's sign
        code = torch.as_tensor(c)[:, 20] & 7
        col = torch.arange(N) != N // 2
        assert torch.equal(torch.isnan(C[M // 2]).cpu()[col], (code == 0)[col])
    assert torch.equal(bad, want)


@pytest.mark.parametrize("which", WHICH)
def test_product_without_inner_dimension(which):
    """K == 0 or alpha == 0: C = beta * C, no operand read; beta == 0 clears a NaN."""
    r = rng(9)
    c0 = r.standard_normal((5, 7)).astype(np.float32)
    for K, alpha in ((0, 1.0), (64, 0.0)):
        args, _ = a_operand(which, r, 5, K, 0, 0)
        B, SB = (torch.as_tensor(v).to(DEV) for v in packed_case(r, 7, K, 255, 255))
        for beta in (0.0, 0.5):
            C = torch.as_tensor(c0 if beta else np.full((5, 7), np.nan, np.float32)).to(DEV)
            product(which, args, B, SB, C, alpha, beta, K)
            assert np.array_equal(C.cpu().numpy(), np.float32(beta) * c0 if beta else np.zeros((5, 7), np.float32))


@pytest.mark.parametrize("which", WHICH)
def test_product_repeats_bit_for_bit_and_on_other_streams(which):
    r = rng(10)
    outs = []
    cases = []
    for (M, N, K) in [(1, 700, 4096), (33, 512, 2048), (512, 1024, 1024)]:
        args, _ = a_operand(which, r, M, K, 0, 0)
        B, SB = (torch.as_tensor(v).to(DEV) for v in packed_case(r, N, K))
        cases.append((args, B, SB, M, N, K))
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        got = []
        with torch.cuda.stream(stream):
            for args, B, SB, M, N, K in cases:
                C = torch.empty((M, N), device=DEV)
                product(which, args, B, SB, C, 1.0, 0.0, K)
                got.append(C)
        stream.synchronize()
        outs.append(got)
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_quantized_products_of_a_training_step():
    """Y = X W^T, dX = G W, dW = G^T X, each operand quantised along the axis its
    product contracts: every one equals the product of the values its packed
    operands stand for, and follows the unquantised one to 4-bit precision."""
    r = rng(11)
    M, N, K = 130, 96, 200
    x, w, g = (torch.as_tensor(r.standard_normal(s)).float().to(DEV) for s in ((M, K), (N, K), (M, N)))

    def pack(t, trans):
        rows, n = (t.shape[1], t.shape[0]) if trans else t.shape
        cs, ss = ll.mx4_shapes(rows, n)
        return ll.mx4_quantize(t, torch.empty(cs, dtype=torch.uint8, device=DEV),
                               torch.empty(ss, dtype=torch.uint8, device=DEV), trans=trans)

    for a, ta, b, tb, inner, exact in ((x, False, w, False, K, x.double() @ w.double().t()),
                                       (g, False, w, True, N, g.double() @ w.double()),
                                       (g, True, x, True, M, g.double().t() @ x.double())):
        (qa, sa), (qb, sb) = pack(a, ta), pack(b, tb)
        C = torch.empty((qa.shape[0], qb.shape[0]), device=DEV)
        ll.gemm_mx4f32_nt(qa, sa, qb, sb, C, K=inner)
        av, bv = values(qa.cpu(), sa.cpu(), inner), values(qb.cpu(), sb.cpu(), inner)
        size = np.abs(av) @ np.abs(bv).T
        assert (np.abs(C.double().cpu().numpy() - av @ bv.T) <= (inner + 8) * HALF_STEP * size).all()
        # a code is off by at most a quarter of its value (6 for 8) or a twelfth of
        # its block's largest: the products' relative distance stays below a half
        assert (C.double() - exact).norm() < 0.5 * exact.norm()


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K,alpha,beta", [(2100, 4200, 544, 1.0, 0.0), (4100, 4200, 1057, 1.5, 0.5), (4352, 4096, 512, 1.0, 0.0)])
def test_product_in_large_tiles(M, N, K, alpha, beta, which):
    """Sizes that fill the chip with 256 x 256 tiles, the last ones in halves, a
    half past the last row, and what K leaves past whole stages."""
    check(which, M, N, K, alpha, beta, seed=12)


@pytest.mark.parametrize("M,N,K,lo,hi", [(2100, 4200, 544, 90, 110), (300, 400, 777, 0, 40), (300, 400, 1024, 130, 160)])
@pytest.mark.parametrize("pad", [0, 3])
def test_product_f16_with_far_scales_in_some_blocks(M, N, K, lo, hi, pad):
    """Scales past binary16 in a few blocks only: in the first or last panel of a
    row, and in what K leaves past whole stages."""
    r = rng(13)
    args, av = a_operand("f16", r, M, K, 13 + 16 * pad, 0)
    c, s = packed_case(r, N, K)
    nb = s.shape[1]
    for n, b in ((0, 0), (N // 2, nb // 2), (N - 1, nb - 1)):
        s[n, b] = r.integers(lo, hi + 1)
    bv = values(c, s, K)
    C = torch.full((M, N), float("nan"), device=DEV)
    product("f16", args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    assert (np.abs(C.double().cpu().numpy() - want) <= (K + 8) * (HALF_STEP * size + 2.0 ** -126)).all()


@pytest.mark.parametrize("which", WHICH)
def test_product_nan_scales_in_large_products(which):
    """NaN blocks in panels of scales: their rows and columns, and no others."""
    M, N, K = 300, 400, 1100
    r = rng(14)
    c, s = packed_case(r, N, K)
    args, av = a_operand(which, r, M, K, 4 if which == "mx4" else 0, 0)
    cols, rows = [0, 127, 399], []
    for n, b in zip(cols, (0, 20, s.shape[1] - 1)):
        s[n, b] = 255
    if which == "mx4":
        rows = [1, 130, 299]
        for m, b in zip(rows, (s.shape[1] - 1, 0, 17)):
            args[1][m, b] = 255
    C = torch.zeros((M, N), device=DEV)
    product(which, args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
    want = torch.zeros((M, N), dtype=torch.bool)
    want[:, cols] = True
    want[rows, :] = True
    assert torch.equal(~torch.isfinite(C).cpu(), want)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("N,K", [(1, 512), (7, 2048), (33, 2049), (300, 4127), (17, 11008), (5, 12001), (3, 40000), (2, 70000)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_product_of_one_row(N, K, pad, shift, which):
    """One row of A: whole turns of 64 blocks and what is left of them, a last block
    cut short, rows of B shared by two waves, A too long for a workgroup's memory."""
    check(which, 1, N, K, 1.0, 0.5 if shift else 0.0, pad, shift, seed=15)


@pytest.mark.parametrize("which", WHICH)
def test_one_row_with_far_scales_and_non_finite_values(which):
    """Every scale byte; an infinity and a NaN of A reach every column, a NaN block of
    B its own column and no other."""
    N, K = 40, 64 * 32 * 3 + 40
    check(which, 1, N, K, lo=0, hi=60, seed=16)
    check(which, 1, N, K, lo=200, hi=230, seed=17)
    r = rng(18)
    c, s = packed_case(r, N, K)
    s[3, 70], s[4, s.shape[1] - 1] = 255, 255
    args, av = a_operand(which, r, 1, K, 0, 0)
    C = torch.zeros((1, N), device=DEV)
    product(which, args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
    want = torch.zeros(N, dtype=torch.bool)
    want[3], want[4] = True, True
    assert torch.equal(torch.isnan(C[0]).cpu(), want)
    if which != "mx4":
        args[0][0, 65] = float("inf")
        product(which, args, torch.as_tensor(c).to(DEV), torch.as_tensor(s).to(DEV), C, 1.0, 0.0, K)
        assert not bool(torch.isfinite(C).any())


SHARED = [(33, 300, 11008), (20, 300, 9001), (8, 70, 8192), (64, 1000, 4100), (5, 16, 30000), (100, 90, 6000)]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", SHARED)
@pytest.mark.parametrize("alpha,beta,pad,shift", [(1.0, 0.0, 0, 0), (1.5, 0.5, 3, 1)])
def test_product_shared_out_over_k(M, N, K, alpha, beta, pad, shift, which):
    """Few tiles and a long K: shares of K through a workspace where the plan finds
    them faster, as the call on the current stream takes one."""
    check(which, M, N, K, alpha, beta, pad, shift, seed=19)


@pytest.mark.parametrize("which", WHICH)
def test_workspace_of_the_c_call(which):
    """The call with a workspace: one too small is refused, a larger one taken, nothing
    past it written, and the result is the call's on the current stream bit for bit."""
    M, N, K = 33, 300, 11008
    r = rng(20)
    args, _ = a_operand(which, r, M, K, 0, 0)
    c, s = (torch.as_tensor(v).to(DEV) for v in packed_case(r, N, K))
    C, D = torch.zeros((M, N), device=DEV), torch.zeros((M, N), device=DEV)
    product(which, args, c, s, C, 1.0, 0.0, K)
    lib = ll.load()
    need = lib.ll_mx4_workspace_size(M, N, K, {"mx4": 0, "f16": 1, "bf16": 2}[which])
    work = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream

    def call(out, p, n):
        b = (c.data_ptr(), c.stride(0), s.data_ptr(), s.stride(0), 0.0, out.data_ptr(), N, p, n, stream)
        if which == "mx4":
            a, sa = args
            return lib.gemm_mx4f32_nt_ws(M, N, K, 1.0, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0), *b)
        f = lib.gemm_f16mx4f32_nt_ws if which == "f16" else lib.gemm_bf16mx4f32_nt_ws
        return f(M, N, K, 1.0, args[0].data_ptr(), args[0].stride(0), *b)

    assert call(D, work.data_ptr(), need - 1) == ll.ERR_INVALID_VALUE
    assert call(D, work.data_ptr() + 4, need) == ll.ERR_INVALID_VALUE
    assert call(D, c.data_ptr(), need) == ll.ERR_INVALID_VALUE
    assert call(D, work.data_ptr(), need + 128) == ll.OK
    assert torch.equal(C, D) and bool((work[need:] == 255).all())
    E = torch.zeros((M, N), device=DEV)
    assert call(E, None, 0) == ll.OK      # without one: another order of the same sums
    assert torch.allclose(E, D, rtol=1e-3, atol=1e-3 * float(D.abs().max()))


def test_shared_products_replay_from_a_graph():
    """A product with a workspace and a norm's input after it, captured and replayed
    with new inputs between the program's own calls."""
    M, N, K = 33, 256, 11008
    r = rng(21)
    A = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    c, s = (torch.as_tensor(v).to(DEV) for v in packed_case(r, N, K))
    C = torch.empty((M, N), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ll.gemm_bf16mx4f32_nt(A, c, s, C)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ll.gemm_bf16mx4f32_nt(A, c, s, C)
    for _ in range(4):
        A.copy_(torch.randn((M, K), device=DEV))
        want = torch.empty_like(C)
        ll.gemm_bf16mx4f32_nt(A, c, s, want)
        C.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("M,N,K", [(1300, 1700, 32), (2100, 1100, 128), (1501, 1603, 201), (1300, 1700, 256)])
@pytest.mark.parametrize("alpha,beta,pad,shift", [(1.0, 0.0, 0, 0), (-1.5, 0.5, 3, 1)])
def test_product_with_a_short_k(M, N, K, alpha, beta, pad, shift, which):
    """Large outputs of a K of one or two turns: one wave to a tile."""
    check(which, M, N, K, alpha, beta, pad, shift, seed=22)
