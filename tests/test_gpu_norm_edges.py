"""The residual norms past the ordinary: more rows than workgroups. Against the formulas
in float64 on the GPU (torch), row slab by row slab.

Tolerances as in test_gpu_norm: 64 half-steps of FP32 (2^-24) of a result's size, the sum
of its terms' magnitudes, and half a step of the output's type, finfo.eps / 2, of its
value."""
import pytest

import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
H32 = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def close(got, want, size, steps, what):
    store = 0.0
    if got.dtype != torch.float32:
        fi = torch.finfo(got.dtype)
        store = fi.eps / 2 * want.abs() * (1 + steps * H32) + fi.smallest_normal * fi.eps / 2
    bad = ~((got.double() - want).abs() <= steps * H32 * size + store)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def r(v, eps):
    return 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)


# a workgroup of several waves takes a second row past 2^20 rows
ROWS, WIDE = (1 << 20) + 4099, 1032


def rows_of_all_sizes(g, dtype):
    """Neighbouring rows differ by up to 2^12, so that another row's sum shows."""
    x = torch.randn((ROWS, WIDE), generator=g, device=DEV, dtype=dtype)
    x *= torch.exp2(torch.randint(-6, 7, (ROWS, 1), generator=g, device=DEV)).to(dtype)
    return x


def test_more_rows_than_workgroups_without_y():
    g = gen(1)
    x, w = rows_of_all_sizes(g, BF), 1 + 0.2 * torch.randn((WIDE,), generator=g, device=DEV)
    h = torch.empty_like(x)
    ll.rmsnorm_residual(None, None, None, 1.0, x, w, None, h)
    for m in range(0, ROWS, 1 << 17):
        v = x[m:m + (1 << 17)].double()
        want = v * r(v, 1e-5) * w.double()
        close(h[m:m + (1 << 17)], want, want.abs(), 64, f"rows from {m}")


def test_more_rows_than_workgroups_without_h():
    g = gen(2)
    x, y = torch.randn((ROWS, WIDE), generator=g, device=DEV, dtype=BF), rows_of_all_sizes(g, torch.float32)
    w, gate = (1 + 0.2 * torch.randn((WIDE,), generator=g, device=DEV) for _ in range(2))
    xo = torch.empty_like(x)
    ll.rmsnorm_residual(y, w, gate, 0.7, x, None, xo, None)
    for m in range(0, ROWS, 1 << 17):
        v = y[m:m + (1 << 17)].double()
        step, xd = 0.7 * gate.double() * w.double() * (v * r(v, 1e-5)), x[m:m + (1 << 17)].double()
        close(xo[m:m + (1 << 17)], xd + step, xd.abs() + step.abs(), 64, f"rows from {m}")


def test_more_rows_than_workgroups_with_both():
    g = gen(3)
    x, y = rows_of_all_sizes(g, BF), rows_of_all_sizes(g, torch.float32)
    w = 1 + 0.2 * torch.randn((WIDE,), generator=g, device=DEV)
    xo, h = torch.empty_like(x), torch.empty_like(x)
    ll.rmsnorm_residual(y, None, None, 0.7, x, w, xo, h)
    for m in range(0, ROWS, 1 << 17):
        v, xd = y[m:m + (1 << 17)].double(), x[m:m + (1 << 17)].double()
        step = 0.7 * (v * r(v, 1e-5))
        out = xd + step
        size = xd.abs() + step.abs()
        close(xo[m:m + (1 << 17)], out, size, 64, f"x', rows from {m}")
        close(h[m:m + (1 << 17)], out * r(out, 1e-5) * w.double(), size * r(out, 1e-5) * w.double().abs(), 64, f"h, rows from {m}")
