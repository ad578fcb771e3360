"""Which kernel a product with a 4-bit operand takes, without a GPU."""
import pytest

import linear_layer_amd as ll

FORMS = (ll.A_MX4, ll.A_F16, ll.A_BF16)
NAMES = {"rows", "rows_shared", "tiny", "short", "tile_256x256", "tile_128x128", "stream_16x16", "stream_32x32",
         "stream_64x64", "stream_16x64", "stream_32x64", "stream_48x64"}


def test_no_kernel_without_work_or_with_bad_arguments():
    k = ll.mx4_chosen_kernel
    assert k(0, 8, 64, 0) == k(4, 0, 64, 0) == k(4, 8, 0, 0) == k(-1, 8, 64, 0) == ""
    assert k(4, 8, 64, 3) == k(4, 8, 64, -1) == ""


@pytest.mark.parametrize("a", FORMS)
def test_kernels_by_shape(a):
    k = lambda *s, **o: ll.mx4_chosen_kernel(*s, a, **o)  # noqa: E731
    assert k(1, 11008, 4096) == "rows" and k(1, 4096, 11008) == "rows_shared"
    assert k(300, 400, 31) == "tiny" and k(5000, 5000, 128) == "short"
    assert k(8192, 8192, 8192) == "tile_256x256" and k(8192, 8192, 8192, aligned=False) == "tile_128x128"
    assert k(33, 4096, 11008).startswith("stream_")
    # the tile kernels take at least a tile, and panels of 16 scales
    for M, N, K in ((127, 8192, 4096), (8192, 127, 4096), (8192, 8192, 511)):
        assert not k(M, N, K).startswith("tile_")
    for M in (1, 2, 17, 100, 300, 5000):
        for N in (1, 16, 300, 11008):
            for K in (1, 31, 32, 100, 500, 5000, 40000):
                assert {k(M, N, K, aligned=al, workspace=w) for al in (True, False) for w in (True, False)} <= NAMES
