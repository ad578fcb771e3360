"""The 16-bit layer's products through each of their kernels (every case asserts the one
it is for), with the reference in float64 on the device by torch, and the calls around
them: captured and replayed, on other streams and at once, far from their base, and a
training step as it is used. Tolerances as in test_gpu_linear16: a sum of n products is
off by at most n steps of 2^-23 of the sum of their magnitudes, and stored with half a
step of its type."""
import threading

import numpy as np
import pytest

import linear16_reference as ref
import linear_layer_amd as ll

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STEP = 2.0 ** -23


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def randn(seed, *shape, t="bf16", scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPES[t])


def close(got, want, size, n, what):
    tol = n * STEP * size
    fi = torch.finfo(got.dtype)
    if got.dtype != torch.float32:
        tol = tol * (1 + fi.eps) + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps / 2
    ok = (got.double() - want).abs() <= tol
    assert ok.all(), f"{what}: {(~ok).sum().item()} of {ok.numel()} outside, first at {(~ok).nonzero()[0].tolist()}"


def both(a, b):
    return a.double() @ b.double(), a.double().abs() @ b.double().abs()


def spans_of(groups, M):
    return ref.bounds(groups, M)


def offsets_of(groups):
    return None if groups is None else torch.tensor(groups, dtype=torch.int32, device=DEV)


def stack(seed, groups, N, K, t, scale):
    w = randn(seed, 1 if groups is None else len(groups) - 1, N, K, t=t, scale=scale)
    return w, (w[0] if groups is None else w)


RAGGED = [0, 700, 700, 1100, 2500, 2560, 4000]

FORWARD = [
    # rows, columns, inner, groups, kernel
    (1, 520, 1000, None, "rows"), (16, 64, 64, None, "rows"), (17, 130, 8192, None, "rows"), (33, 4096, 4104, None, "rows"),
    (64, 200, 2048, None, "rows"), (1, 72, 40, None, "rows"), (40, 136, 512, [0, 1, 1, 30, 38], "rows"),
    (300, 136, 512, [0, 290, 291, 291, 292, 300], "rows"),
    (70, 300, 512, None, "small"), (130, 1000, 72, None, "small"), (500, 260, 136, [0, 3, 300, 500], "small"),
    (1200, 2048, 1024, None, "large"),      # quarters alone
    (1100, 8192, 8200, None, "large"),      # halves alone, of large tiles and of a last row
    (6400, 2000, 1032, None, "large"),       # whole tiles
    (2304, 8192, 512, None, "large"),       # a round and quarters
    (4000, 4096, 1024, RAGGED, "large"),
    (4010, 2056, 2048, [5] + RAGGED[1:], "large"),
]


@pytest.mark.parametrize("case", FORWARD, ids=str)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_forward(case, t):
    M, N, K, groups, kernel = case
    assert ll.linear16_chosen_kernel(ll.L16_FORWARD, M, N, K, 1 if groups is None else len(groups) - 1) == kernel
    x = randn(1, M, K, t=t)
    w, wd = stack(2, groups, N, K, t, K ** -0.5)
    b = randn(3, w.shape[0], N, t="f32")
    r = randn(4, M, N, t=t)
    y = torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV)
    y32 = torch.full((M, N), 7.0, device=DEV)
    q = tuple(torch.zeros(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, N))
    bd = b[0] if groups is None else b
    ll.linear16_nt(x, wd, bd, ll.ACT_RELU, r, y, Z=q, offsets=offsets_of(groups))
    ll.linear16_nt(x, wd, None, ll.ACT_NONE, None, y32, offsets=offsets_of(groups))
    z8 = ll.mx8_dequantize(*q, torch.empty((M, N), device=DEV)).double()
    inside = torch.zeros(M, dtype=torch.bool, device=DEV)
    for g, (a, e) in enumerate(spans_of(groups, M)):
        inside[a:e] = True
        if a == e:
            continue
        z, size = both(x[a:e], w[g].t().contiguous())
        close(y32[a:e], z, size, K, "y in FP32")
        z, size = z + b[g].double(), size + b[g].double().abs()
        want = z.clamp(min=0) + r[a:e].double()
        close(y[a:e], want, size + want.abs(), K + 1, "y")
        err = (K + 1) * STEP * size
        for c in range(0, N, 32):
            top = (z[:, c:c + 32].abs() + err[:, c:c + 32]).amax(1, keepdim=True)
            tol = 2.0 ** -4 * (z[:, c:c + 32].abs() + err[:, c:c + 32]) + 2.0 ** -9 * top / 448 + err[:, c:c + 32]
            assert ((z8[a:e, c:c + 32] - z[:, c:c + 32]).abs() <= tol).all(), c
    assert (y[~inside] == 7).all() and (y32[~inside] == 7).all()


INPUT = [
    (70, 512, 304, None, "small"), (500, 136, 264, [0, 3, 300, 500], "small"),
    (1200, 1024, 2048, None, "large"), (1100, 8200, 8192, None, "large"), (6400, 1032, 2000, None, "large"),
    (4000, 1024, 4096, RAGGED, "large"),
]


@pytest.mark.parametrize("case", INPUT, ids=str)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_grad_input(case, t):
    M, N, K, groups, kernel = case
    assert ll.linear16_chosen_kernel(ll.L16_GRAD_INPUT, M, N, K, 1 if groups is None else len(groups) - 1) == kernel
    dz = randn(1, M, N, t=t)
    w, wd = stack(2, groups, N, K, t, N ** -0.5)
    dx = torch.full((M, K), 7.0, dtype=TYPES[t], device=DEV)
    ll.linear16_grad_input(dz, wd, dx, offsets=offsets_of(groups))
    inside = torch.zeros(M, dtype=torch.bool, device=DEV)
    for g, (a, e) in enumerate(spans_of(groups, M)):
        inside[a:e] = True
        if e > a:
            close(dx[a:e], *both(dz[a:e], w[g]), N, "dx")
    assert (dx[~inside] == 7).all()


WEIGHT = [
    (512, 304, 264, None, "small"), (300, 136, 200, [0, 3, 250, 300], "small"),
    (1200, 2048, 2048, None, "large"), (8191, 1104, 8192, None, "large"), (1032, 6400, 2000, None, "large"),
    (1025, 4096, 2304, [0, 300, 300, 1025], "large"),
]


@pytest.mark.parametrize("case", WEIGHT, ids=str)
@pytest.mark.parametrize("keep", ["", "mx8"])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_grad_weight(case, keep, t):
    M, N, K, groups, kernel = case
    assert ll.linear16_chosen_kernel(ll.L16_GRAD_WEIGHT, M, N, K, 1 if groups is None else len(groups) - 1) == kernel
    dz, x = randn(1, M, N, t=t), randn(2, M, K, t=t)
    xd, xr = x, x.double()
    if keep:
        xd = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, K))
        ll.mx8_quantize(x, *xd)
        xr = ll.mx8_dequantize(*xd, torch.empty((M, K), device=DEV)).double()
    spans = spans_of(groups, M)
    dw = randn(3, len(spans), N, K, t="f32")
    before = dw.double()
    ll.linear16_grad_weight(dz, xd, dw if groups else dw[0], beta=1.0, offsets=offsets_of(groups))
    for g, (a, e) in enumerate(spans):
        want, size = both(dz[a:e].t().contiguous(), xr[a:e])
        close(dw[g], want + before[g], size + before[g].abs(), M + 1, "dw")


@pytest.mark.parametrize("M", [1, 33])
def test_shares_of_the_inner_dimension(M):
    """With a workspace K is shared out where columns are few; equal bits every time, and NaN in
    the workspace before the call goes nowhere."""
    N, K = 200, 11008
    need = ll.linear16_workspace_size(ll.L16_FORWARD, M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    x, w, b = randn(1, M, K), randn(2, N, K, scale=K ** -0.5), randn(3, N, t="f32")
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    s = torch.cuda.current_stream()
    out = []
    for room in (ws, ws, None):
        y = torch.empty((M, N), device=DEV)
        ll.linear16_nt(x, w, b, ll.ACT_NONE, None, y, workspace=room, stream=s)   # without one where None
        out.append(y)
    z, size = both(x, w.t().contiguous())
    for y in out:
        close(y, z + b.double(), size + b.double().abs(), K + 1, "y")
    assert torch.equal(out[0], out[1])
    with pytest.raises(ll.LinearLayerError):
        ll.linear16_nt(x, w, b, ll.ACT_NONE, None, out[0], workspace=ws[:-1])


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 20, 50])
def test_few_rows_at_each_alignment(M, t):
    """X and W with rows on two, four and sixteen bytes, each with each, at inner dimensions that
    end inside a load; the values around the rows are NaN and reach nothing."""
    N = 70
    for K in (8, 197, 200, 1001):
        x, w = randn(1, M, K, t=t), randn(2, N, K, t=t)
        want, size = both(x, w.t())
        for px, sx, pw, sw in ((1, 1, 1, 0), (0, 1, 2, 2), (2, 0, 3, 1), (4, 2, 0, 0), (1, 0, 8 + -K % 8, 0), (-K % 8, 0, 1, 3)):
            def laid(a, pad, shift):
                buf = torch.full((a.shape[0] * (K + pad) + shift + 8,), float("nan"), dtype=TYPES[t], device=DEV)
                v = torch.as_strided(buf, a.shape, (K + pad, 1), shift)
                v.copy_(a)
                return v
            xs, ws = laid(x, px, sx), laid(w, pw, sw)
            y = torch.empty((M, N), device=DEV)
            ll.linear16_nt(xs, ws, None, 0, None, y)
            close(y, want, size, K, "K %d X +%d@%d W +%d@%d" % (K, px, sx, pw, sw))


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(16, 4096, 1024, None), (130, 8200, 520, None), (200, 4096, 136, [0, 3, 3, 190, 198]),
                                  (100, 2047, 333, None)], ids=str)
def test_tiles_in_shares(case, t):
    """Products of few tiles in shares of their contracted axis, with their write-back; rows on 16
    bytes and off them."""
    M, C, N, groups = case      # rows, contracted, columns of the result
    G = 1 if groups is None else len(groups) - 1
    dz = randn(1, M, C, t=t)
    w, wd = stack(2, groups, C, N, t, C ** -0.5)
    need = ll.linear16_workspace_size(ll.L16_GRAD_INPUT, M, C, N, G)
    assert need >= 2 * 4 * M * N
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    dx, dx2, dx3 = (torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV) for _ in range(3))
    s = torch.cuda.current_stream()
    ll.linear16_grad_input(dz, wd, dx, offsets=offsets_of(groups), workspace=ws)
    ll.linear16_grad_input(dz, wd, dx2, offsets=offsets_of(groups))
    ll.linear16_grad_input(dz, wd, dx3, offsets=offsets_of(groups), stream=s)      # whole
    assert torch.equal(dx, dx2)
    for g, (a, e) in enumerate(spans_of(groups, M)):
        for v in (dx, dx3):
            if e > a:
                close(v[a:e], *both(dz[a:e], w[g]), C, "dx")
    outside = torch.ones(M, dtype=torch.bool, device=DEV)
    for a, e in spans_of(groups, M):
        outside[a:e] = False
    assert (dx[outside] == 7).all()
    if M // G > 64:
        wt = w.transpose(1, 2).contiguous()
        assert ll.linear16_workspace_size(ll.L16_FORWARD, M, N, C, G) > 0
        b, r = randn(3, G, N, t="f32"), randn(4, M, N, t=t)
        y = torch.full((M, N), 7.0, dtype=TYPES[t], device=DEV)
        q = tuple(torch.zeros(k, dtype=torch.uint8, device=DEV) for k in ll.mx8_shapes(M, N))
        ll.linear16_nt(dz, wt if groups else wt[0], b if groups else b[0], ll.ACT_RELU, r, y, Z=q, offsets=offsets_of(groups))
        z8 = ll.mx8_dequantize(*q, torch.empty((M, N), device=DEV)).double()
        for g, (a, e) in enumerate(spans_of(groups, M)):
            z, size = both(dz[a:e], w[g])
            z, size = z + b[g].double(), size + b[g].double().abs()
            want = z.clamp(min=0) + r[a:e].double()
            close(y[a:e], want, size + want.abs(), C + 1, "y")
            # half a step of each value's own, or of the smallest code under its block's scale
            err = (C + 1) * STEP * size
            top = torch.nn.functional.pad(z.abs() + err, (0, -N % 32)).view(e - a, -1, 32).amax(2).repeat_interleave(32, 1)[:, :N]
            assert ((z8[a:e] - z).abs() <= 2.0 ** -4 * (z.abs() + err) + 2.0 ** -9 * top / 448 + err).all()


def step(x, ws, b1, dy, offsets, bufs, beta=0.0):
    """A two-layer expert block's training step: forward with its kept inputs, and the way back."""
    w1, w2 = ws
    ll.mx8_quantize(x, *bufs["x8"])
    ll.linear16_nt(x, w1, b1, ll.ACT_SILU, None, bufs["h"], Z=bufs["z8"], offsets=offsets)
    ll.linear16_nt(bufs["h"], w2, None, ll.ACT_NONE, x, bufs["y"], offsets=offsets, workspace=bufs["ws"])
    ll.linear16_grad_weight(dy, bufs["h"], bufs["dw2"], beta=beta, offsets=offsets)
    ll.linear16_grad_input(dy, w2, bufs["dh"], offsets=offsets)
    ll.linear16_grad_act(bufs["dh"], bufs["z8"], ll.ACT_SILU, bufs["dz"], bufs["db1"], offsets=offsets, workspace=bufs["ws"])
    ll.linear16_grad_weight(bufs["dz"], bufs["x8"], bufs["dw1"], beta=beta, offsets=offsets)
    ll.linear16_grad_input(bufs["dz"], w1, bufs["dx"], offsets=offsets)


def step_buffers(M, D, H, G):
    def e(*s, t=torch.bfloat16):
        return torch.zeros(s, dtype=t, device=DEV)
    u8, f = torch.uint8, torch.float32
    return {"x8": tuple(e(*s, t=u8) for s in ll.mx8_shapes(M, D)), "z8": tuple(e(*s, t=u8) for s in ll.mx8_shapes(M, H)),
            "h": e(M, H), "y": e(M, D, t=torch.bfloat16), "dw2": e(G, D, H, t=f), "dh": e(M, H), "dz": e(M, H),
            "db1": e(G, H, t=f), "dw1": e(G, H, D, t=f), "dx": e(M, D),
            "ws": e(max(ll.linear16_grad_act_workspace_size(M, H, G), ll.linear16_workspace_size(ll.L16_FORWARD, M, D, H, G),
                         ll.linear16_workspace_size(ll.L16_GRAD_INPUT, M, D, H, G), 16), t=u8)}


OUTPUTS = ("h", "y", "dw2", "dh", "dz", "db1", "dw1", "dx")


def test_training_step_against_differences():
    """The step's gradients, run together as they are used, against differences of a float64
    forward pass; 8 bits of x and z move them by a few per cent of a sixteenth each."""
    M, D, H, G = 96, 64, 128, 3
    off = [0, 40, 40, 96]
    x, dy = randn(1, M, D), randn(2, M, D)
    w1, w2, b1 = randn(3, G, H, D, scale=D ** -0.5), randn(4, G, D, H, scale=H ** -0.5), randn(5, G, H, t="f32", scale=0.1)
    bufs = step_buffers(M, D, H, G)
    step(x, (w1, w2), b1, dy, offsets_of(off), bufs)

    def loss(xd, w1d, w2d, b1d):
        total = 0.0
        for g, (a, e) in enumerate(spans_of(off, M)):
            z = xd[a:e] @ w1d[g].t() + b1d[g]
            y = (z * torch.sigmoid(z)) @ w2d[g].t()   # (the residual's own gradient is dy, not taken here)
            total = total + (y * dy[a:e].double()).sum()
        return total

    args = [v.double() for v in (x, w1, w2, b1)]
    for name, i in (("dx", 0), ("dw1", 1), ("dw2", 2), ("db1", 3)):
        for seed in range(3):
            v = randn(100 + seed, *args[i].shape, t="f32").double()
            eps = 1e-4
            hi, lo = ([a + s * eps * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
            want = ((loss(*hi) - loss(*lo)) / (2 * eps)).item()
            got = (bufs[name].double() * v).sum().item()
            scale = (bufs[name].double().norm() * v.norm() / v.numel() ** 0.5).item()   # of such a sum with random signs
            # 8 bits: each value off by at most 2^-4, independently: a random sum by 2^-4 of its scale
            assert abs(got - want) <= 2.0 ** -4 * scale * 4, (name, got, want, scale)


def test_step_captured_and_replayed():
    """Two graphs of the step that share a workspace, replayed in turn with new inputs, other
    groups and eager calls between, equal the eager results."""
    M, D, H, G = 300, 256, 520, 4
    w = (randn(1, G, H, D, scale=D ** -0.5), randn(2, G, D, H, scale=H ** -0.5))
    b1, x, dy = randn(3, G, H, t="f32"), randn(4, M, D), randn(5, M, D)
    off = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device=DEV)
    sets = [step_buffers(M, D, H, G) for _ in range(2)]
    sets[1]["ws"] = sets[0]["ws"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            step(x, w, b1, dy, off, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(x, w, b1, dy, off, s)
        graphs.append(g)
    for i, groups in enumerate(([0, 100, 100, 250, 300], [0, 1, 2, 3, 300], [10, 10, 10, 200, 290], [0, 300, 300, 300, 300])):
        x.copy_(randn(10 + i, M, D))
        dy.copy_(randn(20 + i, M, D))
        off.copy_(torch.tensor(groups, dtype=torch.int32))
        eager = step_buffers(M, D, H, G)
        step(x, w, b1, dy, off, eager)
        for s in sets:
            for k in ("h", "y", "dh", "dz", "dx"):
                s[k].zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s in sets:
            for k in OUTPUTS:
                assert torch.equal(s[k], eager[k]), (groups, k)


def test_two_streams_two_threads():
    M, D, H, G = 500, 512, 1024, 3
    off = torch.tensor([0, 200, 210, 500], dtype=torch.int32, device=DEV)
    data, want = [], []
    for i in range(2):
        d = (randn(i, M, D), (randn(10 + i, G, H, D, scale=D ** -0.5), randn(20 + i, G, D, H, scale=H ** -0.5)),
             randn(30 + i, G, H, t="f32"), randn(40 + i, M, D))
        b = step_buffers(M, D, H, G)
        step(*d, off, b)
        data.append(d)
        want.append(b)
    torch.cuda.synchronize()
    got, errors = [step_buffers(M, D, H, G) for _ in range(2)], []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    step(*data[i], off, got[i])
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        for k in OUTPUTS:
            assert torch.equal(got[i][k], want[i][k]), (i, k)


@pytest.mark.parametrize("ld", [1 << 20, (1 << 21) + 8])
def test_far_rows(ld):
    """Rows up to 2^31 elements and more from the base, each wholly in sight of the next; from 2^21
    elements apart they are past the copies' buffers and go through registers."""
    M, K, N = (1 << 31) // ld + 150, 72, 136

    def far(cols, dtype=torch.bfloat16):
        return torch.empty((M - 1) * ld + cols, dtype=dtype, device=DEV).as_strided((M, cols), (ld, 1))

    x, y, dz = far(K), far(N), far(N)
    x.copy_(randn(1, M, K))
    dz.copy_(randn(2, M, N))
    w, b = randn(3, N, K, scale=0.1), randn(4, N, t="f32")
    ll.linear16_nt(x, w, b, ll.ACT_NONE, None, y)
    z, size = both(x.contiguous(), w.t().contiguous())
    close(y, z + b.double(), size + b.double().abs(), K + 1, "y")
    dx = far(K)
    ll.linear16_grad_input(dz, w, dx)
    close(dx, *both(dz.contiguous(), w), N, "dx")
    dw = torch.empty((N, K), device=DEV)
    ll.linear16_grad_weight(dz, x, dw)
    close(dw, *both(dz.t().contiguous(), x.contiguous()), M, "dw")
    out, db = far(N), torch.empty(N, device=DEV)
    ll.linear16_grad_act(dz, y, ll.ACT_RELU, out, db)
    assert torch.equal(out, torch.where(y > 0, dz, torch.zeros_like(dz)))
    q = far(K, torch.uint8), far(3, torch.uint8)
    ll.mx8_quantize(x, *q)
    near = tuple(torch.empty(s, dtype=torch.uint8, device=DEV) for s in ll.mx8_shapes(M, K))
    ll.mx8_quantize(x.contiguous(), *near)
    assert torch.equal(q[0], near[0]) and torch.equal(q[1], near[1])
    got = torch.empty((N, K), device=DEV)
    ll.linear16_grad_weight(dz, q, got)
    want = torch.empty((N, K), device=DEV)
    ll.linear16_grad_weight(dz.contiguous(), near, want)
    xr = ll.mx8_dequantize(*near, torch.empty((M, K), device=DEV))
    for v in (got, want):
        close(v, *both(dz.t().contiguous(), xr), M, "dw from 8 bits")


def test_far_weights():
    """A stack of weights whose last ones lie past 2^31 elements."""
    G, N, K, stride = 3, 264, 136, (1 << 30) + 8 * 1000
    buf = torch.empty(2 * stride + N * K, dtype=torch.bfloat16, device=DEV)
    w = buf.as_strided((G, N, K), (stride, K, 1))
    w.copy_(randn(1, G, N, K, scale=0.1))
    M, off = 500, [0, 200, 230, 500]
    x, dz = randn(2, M, K), randn(3, M, N)
    y, dx = torch.empty((M, N), device=DEV), torch.empty((M, K), device=DEV)
    for m, offs in ((M, off), (30, [0, 10, 11, 30])):      # tiles, and few rows
        ll.linear16_nt(x[:m], w, None, ll.ACT_NONE, None, y[:m], offsets=offsets_of(offs))
        ll.linear16_grad_input(dz[:m], w, dx[:m], offsets=offsets_of(offs))
        for g, (a, e) in enumerate(spans_of(offs, m)):
            close(y[a:e], *both(x[a:e], w[g].t().contiguous()), K, "y")
            close(dx[a:e], *both(dz[a:e], w[g]), N, "dx")
    ll.linear16_grad_weight(dz, x, w, offsets=offsets_of(off))
    for g, (a, e) in enumerate(spans_of(off, M)):
        close(w[g], *both(dz[a:e].t().contiguous(), x[a:e]), M, "dw")
    del buf


def test_many_groups():
    """More groups than a launch has tiles, most of them empty, each kernel."""
    G, N, K = 5000, 40, 64
    w = randn(1, 1, N, K).expand(G, N, K)      # one weight for all
    for M in (900, 70000, 350000):
        r = np.random.default_rng(M)
        off = np.sort(np.concatenate([[0, M], r.integers(0, M, G - 1)])).astype(np.int32)
        x, y = randn(2, M, K), torch.empty((M, N), device=DEV)
        ll.linear16_nt(x, w, None, ll.ACT_NONE, None, y, offsets=torch.as_tensor(off).to(DEV))
        close(y, *both(x, w[0].t().contiguous()), K, M)


def test_no_groups_and_refusals():
    x = randn(1, 5, 64)
    y = torch.full((5, 8), 7.0, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    ll.linear16_nt(x, torch.empty((0, 8, 64), dtype=torch.bfloat16, device=DEV), None, 0, None, y, offsets=none)
    assert (y == 7).all()
    w = randn(2, 8, 64)
    for bad in (lambda: ll.linear16_nt(x, w.half(), None, 0, None, y), lambda: ll.linear16_nt(x, w, None, 9, None, y),
                lambda: ll.linear16_nt(x, w, None, 0, None, y[:4]), lambda: ll.linear16_nt(x, w, y[0], 0, None, y),
                lambda: ll.linear16_nt(x, w, None, 0, y.float(), y), lambda: ll.linear16_nt(x, w, None, 0, None, y, Z=(y, y)),
                lambda: ll.linear16_nt(x, w[None], None, 0, None, y, offsets=none.long()),
                lambda: ll.linear16_nt(x, w, None, 0, None, y, offsets=torch.zeros(2, dtype=torch.int32, device=DEV)),
                lambda: ll.linear16_nt(x, w, None, 0, None, x[:, :8]), lambda: ll.linear16_nt(x.t(), w, None, 0, None, y),
                lambda: ll.linear16_grad_act(y, None, ll.ACT_SILU, y), lambda: ll.linear16_grad_act(y, y, 1, y.float()),
                lambda: ll.linear16_grad_act(y, y, 1, y, torch.empty(9, device=DEV)),
                lambda: ll.linear16_grad_act(y, y, 1, y, torch.empty(8, device=DEV), stream=torch.cuda.current_stream()),
                lambda: ll.linear16_grad_input(y, w, y), lambda: ll.linear16_grad_weight(y, None, w),
                lambda: ll.linear16_grad_weight(y, x, w.t()), lambda: ll.mx8_quantize(x, y, y)):
        with pytest.raises((ValueError, TypeError, ll.LinearLayerError)):
            bad()
    assert (y == 7).all()
