"""The residual norms on the GPU against float64 formulas (norm_reference), which
test_norm_cpu checks against differences; here the gradient meets differences too.

Tolerances. A row's sum takes at most 8 * 3 additions in a thread, 6 across a
wave and 16 across waves; with the few operations around it a result is off by
at most 64 half-steps of FP32 (2^-24) of its size, the sum of its terms'
magnitudes; a gradient chains two such results (128). A sum over M rows adds at
most M additions more. A result stored in 16 bits is rounded once: half a step,
finfo.eps / 2, of its value, or half the smallest subnormal."""
import numpy as np
import pytest

import linear_layer_amd as ll
from norm_reference import forward, gradient

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
H32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def strided(a, pad=0, shift=0):
    buf = torch.full((a.shape[0], shift + a.shape[1] + pad), 7.0, dtype=a.dtype, device=DEV)
    v = buf[:, shift:shift + a.shape[1]]
    v.copy_(a)
    return buf, v


def make(M, N, kind, seed, pad=0, shift=0):
    r = np.random.default_rng(seed)
    t = TYPES[kind]
    d = {}
    for name in ("x", "dxo", "dh"):
        d[name] = torch.as_tensor(r.standard_normal((M, N)) * np.exp(r.standard_normal((1, N)))).to(t)
    d["y"] = torch.as_tensor(r.standard_normal((M, N)) * np.exp(r.standard_normal((1, N)))).float()
    for name in ("w_post", "gate", "w_pre"):
        d[name] = torch.as_tensor(1 + 0.5 * r.standard_normal(N)).float()
    dev = {k: strided(v, pad, shift)[1] if v.dim() == 2 else v.to(DEV) for k, v in d.items()}
    return {k: v.double().numpy() for k, v in d.items()}, dev


def close(got, want, size, steps, what):
    got_t = got
    got = got.detach().double().cpu().numpy()
    fi = torch.finfo(got_t.dtype)
    store = 0.0 if got_t.dtype == torch.float32 else fi.eps / 2 * np.abs(want) * (1 + steps * H32) + fi.smallest_normal * fi.eps / 2
    tol = steps * H32 * size + store
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300))}"


SHAPES = [(1, 1), (2, 7), (5, 64), (3, 511), (4, 512), (2, 513), (7, 1001), (3, 2048), (2, 2049), (9, 4096), (3, 4097),
          (2, 8192), (2, 8193), (1, 16384), (2, 16385), (3, 20001), (700, 96)]


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward(M, N, kind, pad, shift):
    d, dev = make(M, N, kind, M * 31 + N, pad, shift)
    xo, h, sxo, sh = forward(d["y"], d["x"], d["w_post"], d["gate"], 0.7, d["w_pre"], 1e-5)
    (ob, XO), (hb, H) = (strided(torch.zeros((M, N), dtype=TYPES[kind]), pad, shift) for _ in range(2))
    ll.rmsnorm_residual(dev["y"], dev["w_post"], dev["gate"], 0.7, dev["x"], dev["w_pre"], XO, H)
    close(XO, xo, sxo, 64, "x'")
    close(H, h, sh, 64, "h")
    for b, v in ((ob, XO), (hb, H)):     # nothing beside the rows is written
        v.fill_(7.0)
        assert bool((b == 7.0).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N", [(3, 100), (2, 4096), (2, 17000)])
def test_forward_parts(M, N, kind):
    """Without y, vectors or one output; x' over x; each equals the whole."""
    d, dev = make(M, N, kind, 5)
    t = TYPES[kind]
    one = np.ones(N)
    H = torch.empty((M, N), dtype=t, device=DEV)
    ll.rmsnorm_residual(None, None, None, 1.0, dev["x"], dev["w_pre"], None, H)
    _, h, _, sh = forward(None, d["x"], one, one, 1.0, d["w_pre"], 1e-5)
    close(H, h, sh, 64, "h of x alone")
    XO = torch.empty((M, N), dtype=t, device=DEV)
    ll.rmsnorm_residual(dev["y"], None, None, -1.5, dev["x"], None, XO, H)
    xo, h, sxo, sh = forward(d["y"], d["x"], one, one, -1.5, one, 1e-5)
    close(XO, xo, sxo, 64, "x' without vectors")
    close(H, h, sh, 64, "h without vectors")
    X2, H2 = dev["x"].clone(), torch.empty_like(H)
    ll.rmsnorm_residual(dev["y"], None, None, -1.5, X2, None, X2, H2)
    assert torch.equal(X2, XO) and torch.equal(H2, H)
    X3 = torch.empty_like(XO)
    ll.rmsnorm_residual(dev["y"], None, None, -1.5, dev["x"], None, X3, None)
    assert torch.equal(X3, XO)


def test_rows_of_zeros_infinities_and_nan():
    """A row of zeros stays finite through eps; an infinity or NaN stays in its row."""
    M, N = 6, 300
    _, dev = make(M, N, "f32", 6)
    dev["y"][1] = 0
    dev["x"][1] = 0
    dev["y"][2, 7] = float("nan")
    dev["x"][4, 9] = float("inf")
    XO, H = torch.empty((M, N), device=DEV), torch.empty((M, N), device=DEV)
    ll.rmsnorm_residual(dev["y"], dev["w_post"], dev["gate"], 0.7, dev["x"], dev["w_pre"], XO, H)
    assert bool((XO[1] == 0).all()) and bool((H[1] == 0).all())
    assert bool(torch.isnan(XO[2]).all()) and bool(torch.isnan(H[2]).all())
    assert bool(torch.isinf(XO[4, 9])) and not bool(torch.isfinite(H[4, 9]))
    for m in (0, 1, 3, 5):
        assert bool(torch.isfinite(XO[m]).all()) and bool(torch.isfinite(H[m]).all())


def grad_outputs(M, N, kind, pad=0, shift=0):
    t = TYPES[kind]
    (yb, DY), (xb, DX) = strided(torch.zeros((M, N)), pad, shift), strided(torch.zeros((M, N), dtype=t), pad, shift)
    vec = {k: torch.full((N,), float("nan"), device=DEV) for k in ("dgate", "dw_post", "dw_pre")}
    work = torch.full((max(ll.rmsnorm_grad_workspace_size(M, N), 1),), 255, dtype=torch.uint8, device=DEV)
    return yb, DY, xb, DX, vec, work


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N", SHAPES)
def test_gradient(M, N, kind, pad, shift):
    d, dev = make(M, N, kind, M * 37 + N, pad, shift)
    want = gradient(d["dxo"], d["dh"], d["y"], d["x"], d["w_post"], d["gate"], 0.7, d["w_pre"], 1e-5)
    yb, DY, xb, DX, vec, work = grad_outputs(M, N, kind, pad, shift)
    ll.rmsnorm_residual_grad(dev["dxo"], dev["dh"], dev["y"], dev["w_post"], dev["gate"], 0.7, dev["x"], dev["w_pre"],
                             DY, DX, vec["dgate"], vec["dw_post"], vec["dw_pre"], work)
    close(DY, *want["dy"], 128, "dy")
    close(DX, *want["dx"], 128, "dx")
    for k in vec:
        close(vec[k], *want[k], 128 + M, k)
    for b, v in ((yb, DY), (xb, DX)):
        v.fill_(7.0)
        assert bool((b == 7.0).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N", [(4, 130), (600, 260), (3, 17001)])
def test_gradient_parts(M, N, kind):
    """One incoming gradient, no y, no vectors, dx over dx'."""
    d, dev = make(M, N, kind, 8)
    one, zero = np.ones(N), np.zeros((M, N))
    _, DY, _, DX, vec, work = grad_outputs(M, N, kind)
    for dxo, dh in ((True, False), (False, True)):
        want = gradient(d["dxo"] if dxo else zero, d["dh"] if dh else zero, d["y"], d["x"], one, one, 0.7, one, 1e-5)
        ll.rmsnorm_residual_grad(dev["dxo"] if dxo else None, dev["dh"] if dh else None, dev["y"], None, None, 0.7,
                                 dev["x"], None, DY, DX, vec["dgate"], vec["dw_post"], vec["dw_pre"], work)
        close(DY, *want["dy"], 128, "dy")
        close(DX, *want["dx"], 128, "dx")
        for k in vec:
            close(vec[k], *want[k], 128 + M, k)
    # without y: the norm before the first block
    rx = 1 / np.sqrt((d["x"] ** 2).mean(1, keepdims=True) + 1e-5)
    n, k = d["x"] * rx, d["dh"] * d["w_pre"]
    total = rx * (k - n * (k * n).mean(1, keepdims=True))
    size = rx * (np.abs(k) + np.abs(n) * np.abs(k * n).mean(1, keepdims=True))
    ll.rmsnorm_residual_grad(None, dev["dh"], None, None, None, 1.0, dev["x"], dev["w_pre"], None, DX, None, None,
                             vec["dw_pre"], work)
    close(DX, total, size, 128, "dx without y")
    close(vec["dw_pre"], (d["dh"] * n).sum(0), np.abs(d["dh"] * n).sum(0), 128 + M, "dw_pre without y")
    # in place, and equal to the same call out of place
    ll.rmsnorm_residual_grad(dev["dxo"], dev["dh"], dev["y"], None, dev["gate"], 0.7, dev["x"], dev["w_pre"], DY, DX,
                             None, None, None, work)
    over = dev["dxo"].clone()
    ll.rmsnorm_residual_grad(over, dev["dh"], dev["y"], None, dev["gate"], 0.7, dev["x"], dev["w_pre"], None, over,
                             None, None, None, work)
    assert torch.equal(over, DX)


def test_gradient_without_rows():
    N = 70
    e = torch.empty((0, N), device=DEV)
    vec = [torch.full((N,), float("nan"), device=DEV) for _ in range(3)]
    ll.rmsnorm_residual_grad(e, e, e, None, None, 1.0, e, None, e, e, *vec, None)
    for v in vec:
        assert bool((v == 0).all())


def test_gradient_against_differences():
    """Directional differences of the float64 forward at the inputs the GPU saw:
    the step 1e-5 of inputs near 1 leaves about 1e-9 of the loss's size; the FP32
    gradient's own error is 128 half-steps of its terms' sizes."""
    M, N, alpha = 5, 40, 0.7
    d, dev = make(M, N, "f32", 9)
    _, DY, _, DX, vec, work = grad_outputs(M, N, "f32")
    ll.rmsnorm_residual_grad(dev["dxo"], dev["dh"], dev["y"], dev["w_post"], dev["gate"], alpha, dev["x"], dev["w_pre"],
                             DY, DX, vec["dgate"], vec["dw_post"], vec["dw_pre"], work)
    got = {"y": DY, "x": DX, "gate": vec["dgate"], "w_post": vec["dw_post"], "w_pre": vec["dw_pre"]}
    size = gradient(d["dxo"], d["dh"], d["y"], d["x"], d["w_post"], d["gate"], alpha, d["w_pre"], 1e-5)
    r = np.random.default_rng(10)

    def loss(v):
        xo, h, _, _ = forward(v["y"], v["x"], v["w_post"], v["gate"], alpha, v["w_pre"], 1e-5)
        return (d["dxo"] * xo).sum() + (d["dh"] * h).sum()

    for name in got:
        way = r.standard_normal(d[name].shape)
        diff = (loss({**d, name: d[name] + 1e-5 * way}) - loss({**d, name: d[name] - 1e-5 * way})) / 2e-5
        terms = (size["d" + name][1] * np.abs(way)).sum()
        assert abs(diff - (got[name].double().cpu().numpy() * way).sum()) <= (128 + M) * H32 * terms + 1e-7 * terms


def test_norms_on_other_streams_and_in_a_graph():
    """Forward and gradient captured together and replayed with new inputs between
    the program's own eager work: every replay equals the eager result bit for bit."""
    M, N = 65, 1000
    _, dev = make(M, N, "bf16", 11)
    t = torch.bfloat16
    XO, H, DX = (torch.empty((M, N), dtype=t, device=DEV) for _ in range(3))
    _, DY, _, _, vec, work = grad_outputs(M, N, "bf16")

    def step():
        ll.rmsnorm_residual(dev["y"], dev["w_post"], dev["gate"], 0.7, dev["x"], dev["w_pre"], XO, H)
        ll.rmsnorm_residual_grad(dev["dxo"], dev["dh"], dev["y"], dev["w_post"], dev["gate"], 0.7, dev["x"], dev["w_pre"],
                                 DY, DX, vec["dgate"], vec["dw_post"], vec["dw_pre"], work)

    outs = [XO, H, DX, DY, *vec.values()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for k in range(4):
        dev["x"].copy_(torch.randn((M, N), device=DEV))
        dev["y"].copy_(torch.randn((M, N), device=DEV))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
