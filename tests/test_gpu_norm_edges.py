"""The residual norms past the ordinary: more rows than workgroups, no y and no eps.
Against the formulas in float64 on the GPU (torch), slab by slab.

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


@pytest.mark.parametrize("M,N", [(3, 100), (40, 600), (5, 4096), (2, 9001)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_gradient_without_y_takes_nothing_from_its_norm(M, N, dtype, eps):
    """x' = x: neither the norm of an absent y (1 / 0 where eps is 0) nor w_post, gate
    and alpha, whatever they hold, have a part in dx and dw_pre. A chain of two results
    each 64 half-steps off: 128; a sum over M rows M more."""
    g = gen(4)
    x, dxo, dh = (torch.randn((M, N), generator=g, device=DEV).to(dtype) for _ in range(3))
    w = 1 + 0.2 * torch.randn((N,), generator=g, device=DEV)
    xd, kd = x.double(), dh.double() * w.double()
    rx = r(xd, eps)
    n = xd * rx
    total = dxo.double() + rx * (kd - n * (kd * n).mean(1, keepdim=True))
    size = dxo.double().abs() + rx * (kd.abs() + n.abs() * (kd * n).abs().mean(1, keepdim=True))
    sums, sum_size = (dh.double() * n).sum(0), (dh.double() * n).abs().sum(0)
    work = torch.empty((ll.rmsnorm_grad_workspace_size(M, N),), dtype=torch.uint8, device=DEV)
    far = torch.full((N,), float("nan"), device=DEV)
    far[::2] = float("inf")
    for w_post, gate, alpha in ((None, None, 1.0), (far, None, 1.0), (None, far, 0.7), (None, None, float("inf"))):
        dx, dw = torch.full_like(x, -7.0), torch.full((N,), -7.0, device=DEV)
        ll.rmsnorm_residual_grad(dxo, dh, None, w_post, gate, alpha, x, w, None, dx, None, None, dw, work, eps=eps)
        close(dx, total, size, 128, "dx")
        close(dw, sums, sum_size, 128 + M, "dw_pre")


def test_gradient_of_a_row_past_a_launch():
    """More columns than the finishing launch has work items for. x is 1 and -1 and dh
    whole numbers, so that the sums over the row are exact but for its last additions,
    and the ordinary 128 half-steps hold."""
    N = 2 ** 28 + 1000
    g = gen(5)
    x = (2 * torch.randint(0, 2, (1, 1009), generator=g, device=DEV) - 1).to(BF).repeat(1, N // 1009 + 1)[:, :N]
    dh = torch.randint(-3, 4, (1, 997), generator=g, device=DEV).to(BF).repeat(1, N // 997 + 1)[:, :N]
    dx, dw = torch.full((1, N), 7.0, dtype=BF, device=DEV), torch.full((N,), float("nan"), device=DEV)
    work = torch.empty((ll.rmsnorm_grad_workspace_size(1, N),), dtype=torch.uint8, device=DEV)
    ll.rmsnorm_residual_grad(None, dh, None, None, None, 1.0, x, None, None, dx, None, None, dw, work, eps=0.0)
    mean = (dh.double() * x.double()).mean()
    for c in range(0, N, 1 << 26):
        xs, ds = x[:, c:c + (1 << 26)].double(), dh[:, c:c + (1 << 26)].double()
        close(dx[:, c:c + (1 << 26)], ds - xs * mean, ds.abs() + xs.abs() * mean.abs(), 128, f"dx from {c}")
        close(dw[c:c + (1 << 26)], (ds * xs)[0], (ds * xs)[0].abs(), 129, f"dw_pre from {c}")


def test_gradient_without_rows_is_zero_whatever_the_vectors_hold():
    """The C call, with pointers to matrices of no rows."""
    N = 70
    m, bad = torch.empty((1, N), device=DEV), torch.full((N,), float("inf"), device=DEV)
    vec = [torch.full((N,), float("nan"), device=DEV) for _ in range(3)]
    p, b = m.data_ptr(), bad.data_ptr()
    st = ll.load().rmsnorm_residual_grad(0, N, ll.TYPE_F32, p, N, p, N, p, N, b, b, 0.5, p, N, b, 1e-5, p, N, p, N,
                                         *(v.data_ptr() for v in vec), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == ll.OK
    for v in vec:
        assert bool((v == 0).all())
