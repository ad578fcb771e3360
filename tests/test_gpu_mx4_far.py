"""The 4-bit operators at the far end of the sizes: launches that have to be cut into
several. Inputs repeat a short pattern, whose outcome the plain float64 implementation
gives; the whole output is compared with it."""
import numpy as np
import pytest

import linear_layer_amd as ll
from mx4_reference import quantize

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
