"""The 4-bit entry points without a GPU: refusals before anything is enqueued,
the reference implementation's own pins, and the binding's checks."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import GRID, quantize, values

E = ll.ERR_INVALID_VALUE
FINE = (ll.OK, ll.ERR_NO_DEVICE, ll.ERR_UNSUPPORTED_ARCH)
PX, PC, PS, PB, PT, PO = (0x10000000 * i for i in range(1, 7))   # addresses nothing may touch


def no_device():
    import torch
    return not torch.cuda.is_available()


def quant(M=4, K=64, type=0, X=PX, ldx=None, trans=0, codes=PC, ldq=None, scales=PS, lds=None):
    n = M if trans else K
    return ll.load().mx4_quantize(M, K, type, X, max(K, 1) if ldx is None else ldx, trans, codes,
                                  max((n + 1) // 2, 1) if ldq is None else ldq, scales,
                                  max((n + 31) // 32, 1) if lds is None else lds, None)


def dequant(M=4, K=64, codes=PC, ldq=None, scales=PS, lds=None, type=0, Y=PX, ldy=None):
    return ll.load().mx4_dequantize(M, K, codes, max((K + 1) // 2, 1) if ldq is None else ldq, scales,
                                    max((K + 31) // 32, 1) if lds is None else lds, type, Y,
                                    max(K, 1) if ldy is None else ldy, None)


def gemm(M=4, N=8, K=64, alpha=1.0, A=PX, lda=None, SA=PS, ldsa=None, B=PB, ldb=None, SB=PT, ldsb=None, beta=0.0,
         C=PO, ldc=None):
    q, s = max((K + 1) // 2, 1), max((K + 31) // 32, 1)
    pick = lambda v, d: d if v is None else v  # noqa: E731
    return ll.load().gemm_mx4f32_nt(M, N, K, alpha, A, pick(lda, q), SA, pick(ldsa, s), B, pick(ldb, q), SB,
                                    pick(ldsb, s), beta, C, pick(ldc, max(N, 1)), None)


def gemm16(name, M=4, N=8, K=64, alpha=1.0, A=PX, lda=None, B=PB, ldb=None, SB=PT, ldsb=None, beta=0.0, C=PO, ldc=None):
    pick = lambda v, d: d if v is None else v  # noqa: E731
    return getattr(ll.load(), name)(M, N, K, alpha, A, pick(lda, max(K, 1)), B, pick(ldb, max((K + 1) // 2, 1)), SB,
                                    pick(ldsb, max((K + 31) // 32, 1)), beta, C, pick(ldc, max(N, 1)), None)


@pytest.mark.parametrize("trans", [0, 1])
def test_quantize_refusals(trans):
    q = lambda **k: quant(trans=trans, **k)  # noqa: E731
    assert q(M=-1) == E and q(K=-1) == E and q(type=3) == E and q(type=-1) == E
    assert quant(trans=2) == E
    assert q(ldx=63) == E
    assert q(ldq=1) == E and q(lds=0) == E
    assert q(X=None) == E and q(codes=None) == E and q(scales=None) == E
    assert q(X=PX + 2) == E and q(type=1, X=PX + 1) == E
    assert q(codes=PX + 16) == E and q(scales=PX) == E and q(scales=PC + 1) == E
    assert q(M=0, X=None, codes=None, scales=None) == ll.OK
    assert q(K=0, X=None, codes=None, scales=None) == ll.OK


def test_dequantize_refusals():
    assert dequant(M=-1) == E and dequant(K=-1) == E and dequant(type=3) == E
    assert dequant(ldy=63) == E and dequant(ldq=31) == E and dequant(lds=1) == E
    assert dequant(Y=None) == E and dequant(codes=None) == E and dequant(scales=None) == E
    assert dequant(Y=PX + 1) == E and dequant(Y=PC - 4) == E
    assert dequant(M=0, codes=None, scales=None, Y=None) == ll.OK
    assert dequant(K=0, codes=None, scales=None, Y=None) == ll.OK


def test_product_refusals():
    for k in ("M", "N", "K"):
        assert gemm(**{k: -1}) == E
    assert gemm(lda=31) == E and gemm(ldb=31) == E and gemm(ldsa=1) == E and gemm(ldsb=1) == E and gemm(ldc=7) == E
    assert gemm(K=65, lda=32) == E and gemm(K=65, ldsa=2) == E
    for k in ("A", "SA", "B", "SB", "C"):
        assert gemm(**{k: None}) == E
    assert gemm(C=PO + 2) == E
    for p in (PX, PS, PB, PT):
        assert gemm(C=p) == E
    assert gemm(M=0, A=None, SA=None, C=None) == ll.OK and gemm(N=0, B=None, SB=None, C=None) == ll.OK


@pytest.mark.parametrize("name", ["gemm_f16mx4f32_nt", "gemm_bf16mx4f32_nt"])
def test_product_16_refusals(name):
    f = lambda **k: gemm16(name, **k)  # noqa: E731
    for k in ("M", "N", "K"):
        assert f(**{k: -1}) == E
    assert f(lda=63) == E and f(ldb=31) == E and f(ldsb=1) == E and f(ldc=7) == E
    for k in ("A", "B", "SB", "C"):
        assert f(**{k: None}) == E
    assert f(A=PX + 1) == E and f(C=PO + 1) == E
    for p in (PX + 8, PB, PT):
        assert f(C=p) == E
    assert f(M=0, A=None, C=None) == ll.OK


def test_good_arguments_reach_the_device_check():
    """Only where there is no device: with one, these would run on made-up addresses."""
    if not no_device():
        pytest.skip("a device is visible")
    assert quant() in FINE and quant(trans=1) in FINE and dequant() in FINE and gemm() in FINE
    for name in ("gemm_f16mx4f32_nt", "gemm_bf16mx4f32_nt"):
        assert gemm16(name) in FINE
    # neither operand is read when alpha is 0
    assert gemm(alpha=0.0, A=None, SA=None, B=None, SB=None) in FINE


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(TypeError):
        ll.mx4_quantize(torch.zeros((4, 64), dtype=torch.float64), u8(4, 32), u8(4, 2))
    with pytest.raises(ValueError):
        ll.mx4_quantize(torch.zeros((4, 64)), u8(4, 32), u8(4, 2))        # host tensors
    with pytest.raises(TypeError):
        ll.gemm_bf16mx4f32_nt(torch.zeros((4, 64), dtype=torch.float16), u8(8, 32), u8(8, 2), torch.zeros(4, 8))
    assert ll.mx4_shapes(3, 65) == ((3, 33), (3, 3))


def test_reference_pins():
    """The reference implementation on blocks worked out by hand."""
    x = np.zeros((4, 33))
    x[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]       # top 6: scale 1; ties go to even codes
    x[1, :4] = [0.1, -7.9, 4, 6.4]                            # top 7.9: scale 1, 7.9 and 6.4 to 6
    x[2, :2] = [8, 1]                                         # top 8: scale 2
    x[3, 32] = -3.0                                           # a block of one value: top 3, scale 1/2
    codes, scales = quantize(x)
    assert codes.shape == (4, 17) and scales.shape == (4, 2)
    v = values(codes, scales, 33)
    assert list(v[0, :8]) == [6, 4, 4, 2, 2, 1, 1, 0]
    assert list(v[1, :4]) == [0, -6, 4, 6] and scales[1, 0] == 127
    assert list(v[2, :2]) == [8, 1] and scales[2, 0] == 128
    assert v[3, 32] == -3.0 and scales[3, 1] == 126 and scales[3, 0] == 0
    y = np.array([[np.inf] + [1.0] * 31 + [np.nan]])
    codes, scales = quantize(y)
    assert list(scales[0]) == [255, 255] and not codes.any() and np.isnan(values(codes, scales, 33)).all()
    # a value of the grid comes back as itself
    g = np.concatenate([GRID, -GRID, GRID, -GRID])[None, :]
    assert np.array_equal(values(*quantize(g), 32), g)


def test_workspace_size_and_refusals():
    lib = ll.load()
    size = lib.ll_mx4_workspace_size
    assert size(-1, 8, 64, 0) == -1 and size(4, -1, 64, 0) == -1 and size(4, 8, -1, 0) == -1
    assert size(4, 8, 64, 3) == -1 and size(4, 8, 64, -1) == -1
    assert size(0, 8, 64, 0) == 0 and size(1, 11008, 4096, 2) == 0 and size(8192, 8192, 8192, 0) == 0
    assert size(33, 4096, 11008, 1) > 0 and size(33, 4096, 11008, 1) % (33 * 4096 * 4) == 0
    for a in (0, 1, 2):
        for M in (1, 3, 17, 100, 1000):
            for N in (16, 500, 11008):
                for K in (1, 31, 100, 5000, 100000):
                    assert 0 <= size(M, N, K, a) <= 64e6
    q, s = 32, 2
    call = lambda ws, n: lib.gemm_mx4f32_nt_ws(4, 8, 64, 1.0, PX, q, PS, s, PB, q, PT, s, 0.0, PO, 8, ws, n, None)  # noqa: E731
    assert call(PX, 256) == E and call(PO, 256) == E and call(PC + 8, 256) == E and call(PC, -1) == E
    if no_device():
        assert call(PC, 256) in FINE and call(None, 0) in FINE
