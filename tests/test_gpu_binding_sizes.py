"""Sizes and row strides past a C int: the binding says so. Passed on as they are,
their lower 32 bits would be taken for them."""
import pytest

import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FAR = 2 ** 32 + 64   # its lower 32 bits are a stride that the shapes below allow


@pytest.fixture(scope="module")
def big():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield torch.zeros(4 * (FAR + 256), dtype=torch.uint8, device=DEV)
    torch.cuda.empty_cache()


def far(big, dtype, cols):
    """Two rows of `cols` values, FAR apart."""
    return big.view(dtype)[:FAR + cols].as_strided((2, cols), (FAR, 1))


def near(dtype, rows, cols):
    return torch.zeros((rows, cols), dtype=dtype, device=DEV)


def test_row_strides_past_an_int(big):
    f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8
    refused = [
        lambda: ll.gemm_f32(far(big, f32, 64), near(f32, 64, 8), near(f32, 2, 8)),
        lambda: ll.gemm_f32(near(f32, 2, 64), near(f32, 64, 8), far(big, f32, 8)),
        lambda: ll.gemm_bf16f32_batched(far(big, bf, 64)[None], near(bf, 64, 8)[None], near(f32, 2, 8)[None]),
        lambda: ll.linear_bias_act(far(big, f32, 64), near(f32, 64, 8), None, 0, near(f32, 2, 8)),
        lambda: ll.mx4_quantize(far(big, bf, 64), near(u8, 2, 32), near(u8, 2, 2)),
        lambda: ll.mx4_quantize(near(bf, 2, 64), far(big, u8, 32), near(u8, 2, 2)),
        lambda: ll.mx4_quantize(near(bf, 2, 64), near(u8, 2, 32), far(big, u8, 2)),
        lambda: ll.mx4_dequantize(near(u8, 2, 32), near(u8, 2, 2), far(big, bf, 64)),
        lambda: ll.gemm_mx4f32_nt(far(big, u8, 32), near(u8, 2, 2), near(u8, 2, 32), near(u8, 2, 2), near(f32, 2, 2)),
        lambda: ll.gemm_bf16mx4f32_nt(near(bf, 2, 64), far(big, u8, 32), near(u8, 2, 2), near(f32, 2, 2)),
        lambda: ll.rmsnorm_residual(None, None, None, 1.0, far(big, f32, 64), None, None, near(f32, 2, 64)),
        lambda: ll.rmsnorm_residual(None, None, None, 1.0, near(f32, 2, 64), None, None, far(big, f32, 64)),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError, match="2147483647"):
            call()
            pytest.fail(f"call {i} was taken")
    # one row has no stride
    one = far(big, f32, 64)[:1]
    ll.rmsnorm_residual(None, None, None, 1.0, one, None, None, near(f32, 1, 64))


def test_sizes_past_an_int(big):
    with pytest.raises(ValueError, match="2147483647"):
        ll.mx4_quantize(big.view(torch.bfloat16)[:2 ** 31, None], near(torch.uint8, 1, 1), near(torch.uint8, 1, 1))
    with pytest.raises(ValueError, match="2147483647"):
        ll.rmsnorm_residual(None, None, None, 1.0, big.view(torch.bfloat16)[None, :2 ** 31], None, None, big.view(torch.bfloat16)[None, :2 ** 31])
    for M, N in ((2 ** 32 + 4, 64), (4, 2 ** 32 + 64)):
        with pytest.raises(ValueError, match="2147483647"):
            ll.rmsnorm_grad_workspace_size(M, N)
