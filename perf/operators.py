"""The low-precision linear block's operators as measured work.

Five operators, each through the package's public calls:

* ``fake_quantize``: ``mx4_quantize`` then ``mx4_dequantize``. A tensor is put
  into microscaled 4-bit floating point (blocks of 32 values along a row, E2M1
  elements, one E8M0 scale a block) and read back as the values it stands for.
  ``trans`` quantises along the columns and gives the transposed tensor, as the
  products of a backward pass need it.
* ``product_mx4``: ``gemm_mx4f32_nt``, C = A * B^T with both operands in that format.
* ``product_16``: ``gemm_bf16mx4f32_nt`` / ``gemm_f16mx4f32_nt``, C = A * B^T with 16-bit
  activations and the weight B in that format.
* ``norm``: ``rmsnorm_residual``, the residual step between two blocks:
  x' = x + alpha * gate * rms(y) * w_post, h = rms(x') * w_pre.
* ``norm_grad``: its gradient, to y, x, gate, w_post and w_pre.

The listed sizes are those of the package's own workloads: the fully-connected
layer 4096 -> 11008 with 1 and 2047 rows, and the 8192-cubed product.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
EPS = 1e-5


def listed():
    return [
        # activations of 8192 tokens put into 4 bits before a wide product
        {"name": "quant_bf16_8192x8192", "op": "fake_quantize", "M": 8192, "K": 8192, "type": "bf16", "trans": False, "pad": 0},
        # the gradient of a ragged batch, quantised along the batch for the weight's gradient
        {"name": "quant_t_f32_2047x11008", "op": "fake_quantize", "M": 2047, "K": 11008, "type": "f32", "trans": True, "pad": 0},
        # one token through a 4096 -> 11008 layer: latency and weight reading
        {"name": "mx4_1x11008x4096", "op": "product_mx4", "M": 1, "N": 11008, "K": 4096, "pad": 0},
        # a ragged prompt through the same layer
        {"name": "mx4_2047x11008x4096", "op": "product_mx4", "M": 2047, "N": 11008, "K": 4096, "pad": 0},
        # the largest product
        {"name": "mx4_8192x8192x8192", "op": "product_mx4", "M": 8192, "N": 8192, "K": 8192, "pad": 0},
        # one token, activations kept in bfloat16
        {"name": "bf16mx4_1x11008x4096", "op": "product_16", "M": 1, "N": 11008, "K": 4096, "type": "bf16", "pad": 0},
        # a decode step of 33 requests through the layer's way back, in binary16
        {"name": "f16mx4_33x4096x11008", "op": "product_16", "M": 33, "N": 4096, "K": 11008, "type": "f16", "pad": 0},
        # a ragged prompt, activations kept in bfloat16
        {"name": "bf16mx4_2047x11008x4096", "op": "product_16", "M": 2047, "N": 11008, "K": 4096, "type": "bf16", "pad": 0},
        # between two blocks, a decode step of 4 requests: latency
        {"name": "norm_f16_4x4096", "op": "norm", "M": 4, "N": 4096, "type": "f16", "pad": 0},
        # between two blocks, a prompt of 8192 tokens
        {"name": "norm_bf16_8192x4096", "op": "norm", "M": 8192, "N": 4096, "type": "bf16", "pad": 0},
        # a training step's residual between two blocks
        {"name": "normgrad_bf16_8191x4096", "op": "norm_grad", "M": 8191, "N": 4096, "type": "bf16", "pad": 0},
        # a small odd one in fp32, rows one value apart from a vector's alignment
        {"name": "normgrad_f32_129x1001", "op": "norm_grad", "M": 129, "N": 1001, "type": "f32", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fake_quantize", "product_mx4", "product_mx4", "product_16", "product_16", "norm", "norm_grad"])
    pad = rng.choice([0, 0, 0, 1, 16])
    if op == "fake_quantize":
        M, K = _log(rng, 1, 8192), _log(rng, 32, 11008)
        M = min(M, 8192 * 8192 // K)
        return {"op": op, "M": M, "K": K, "type": rng.choice(list(TYPES)), "trans": rng.random() < 0.4, "pad": pad}
    if op in ("product_mx4", "product_16"):
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 11008), _log(rng, 32, 11008)
        if rng.random() < 0.6:   # whole blocks, as trained models have them
            K = (K + BLOCK - 1) // BLOCK * BLOCK
        N = max(1, min(N, 8192 ** 3 // (M * K)))
        c = {"op": op, "M": M, "N": N, "K": K, "pad": pad}
        if op == "product_16":
            c["type"] = rng.choice(["f16", "bf16"])
        return c
    M, N = _log(rng, 1, 8192), _log(rng, 64, 8192)
    return {"op": op, "M": M, "N": N, "type": rng.choice(list(TYPES)), "pad": pad}


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _rows(rows, cols, pad, dtype):
    """rows x cols whose rows lie cols + pad elements apart."""
    return torch.zeros((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _activations(g, rows, cols, dtype, pad):
    """Normal values with channels of different size, as hidden states have them."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(0.7 * torch.randn((cols,), generator=g, device=DEV))
    out = _rows(rows, cols, pad, dtype)
    out.copy_(x)
    return out


def _packed(g, rows, K, pad, scale):
    """A tensor in 4 bits as a checkpoint or a quantiser hands it over: codes as
    normal values give them, and scales that vary from block to block."""
    nb = -(-K // BLOCK)
    v = torch.randn((rows, nb * BLOCK), generator=g, device=DEV)
    v[:, K:] = 0
    b = v.view(rows, nb, BLOCK)
    b *= (2.8 / b.abs().amax(dim=2, keepdim=True).clamp_min(1e-3)) * (1.45 + 0.6 * torch.rand((rows, nb, 1), generator=g, device=DEV))
    a = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=DEV)
    for step in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a > step
    code += 8 * (v < 0)
    codes = _rows(rows, (K + 1) // 2, pad, torch.uint8)
    codes.copy_((code[:, 0::2] | (code[:, 1::2] << 4))[:, :(K + 1) // 2])
    scales = _rows(rows, nb, pad, torch.uint8)
    scales.copy_(torch.randint(scale - 2, scale + 3, (rows, nb), generator=g, device=DEV))
    return codes, scales


def prepare(case, seed):
    g, pad, op = _gen(seed), case["pad"], case["op"]
    s = dict(case)
    M = case["M"]
    if op == "fake_quantize":
        K, t = case["K"], TYPES[case["type"]]
        s["x"] = _activations(g, M, K, t, pad)
        r, c = (K, M) if case["trans"] else (M, K)
        s["codes"], s["scales"] = _rows(r, (c + 1) // 2, pad, torch.uint8), _rows(r, -(-c // BLOCK), pad, torch.uint8)
        s["out"] = torch.empty((r, c), dtype=t, device=DEV)
    elif op in ("product_mx4", "product_16"):
        N, K = case["N"], case["K"]
        if op == "product_mx4":
            s["a"], s["sa"] = _packed(g, M, K, pad, 126)
        else:
            s["a"] = _activations(g, M, K, TYPES[case["type"]], pad)
        s["b"], s["sb"] = _packed(g, N, K, pad, 119)
        s["out"] = torch.empty((M, N), device=DEV)
    else:
        N, t = case["N"], TYPES[case["type"]]
        s["y"] = _activations(g, M, N, torch.float32, pad)
        s["x"] = _activations(g, M, N, t, pad)
        for name in ("w_post", "w_pre"):
            s[name] = 1 + 0.2 * torch.randn((N,), generator=g, device=DEV)
        s["gate"] = 0.5 + 0.3 * torch.randn((N,), generator=g, device=DEV)
        s["alpha"] = 0.7
        if op == "norm":
            s["xo"], s["h"] = torch.empty((M, N), dtype=t, device=DEV), torch.empty((M, N), dtype=t, device=DEV)
        else:
            s["dxo"] = _activations(g, M, N, t, pad)
            s["dh"] = _activations(g, M, N, t, pad)
            s["dy"], s["dx"] = torch.empty((M, N), device=DEV), torch.empty((M, N), dtype=t, device=DEV)
            for name in ("dgate", "dw_post", "dw_pre"):
                s[name] = torch.empty((N,), device=DEV)
            # room for the partial sums over rows, as a training program keeps it
            s["work"] = torch.empty((4 * 2 * N * 1024,), dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms ----------------------------------------------------------

def _table():
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)


def _decode(codes, scales, K):
    """The values that codes and scales stand for, in 32 bits."""
    both = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)[:, :K]
    v = _table()[both.long()]
    e = torch.repeat_interleave(scales.int() - 127, BLOCK, dim=1)[:, :K]
    return torch.ldexp(v, e)


def _plain_quantize(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.zeros((rows, nb * BLOCK), device=DEV)
    v[:, :cols] = x
    v = v.view(rows, nb, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)   # floor(log2(top)) - 2
    e = torch.where(top == 0, -127, e)
    a = torch.ldexp(v.abs(), -e)
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    q = torch.ldexp(_table()[code.long()], e)
    q = torch.where(v < 0, -q, q)
    return q.reshape(rows, -1)[:, :cols].to(x.dtype).contiguous()


def _rms(v):
    return torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)


def _plain_norm(s):
    x, y = s["x"].float(), s["y"]
    xo = x + s["alpha"] * s["gate"] * (y * _rms(y) * s["w_post"])
    h = xo * _rms(xo) * s["w_pre"]
    return xo.to(s["x"].dtype), h.to(s["x"].dtype)


def _plain_norm_grad(s):
    x, y, dxo, dh = s["x"].float(), s["y"], s["dxo"].float(), s["dh"].float()
    ry = _rms(y)
    u = y * ry
    t = s["alpha"] * s["gate"] * s["w_post"]
    xo = x + t * u
    rx = _rms(xo)
    n = xo * rx
    dn = dh * s["w_pre"]
    dx = dxo + rx * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    du = dx * t
    dy = ry * (du - u * (du * u).mean(dim=1, keepdim=True))
    both = (dx * u).sum(dim=0)
    return {"dy": dy, "dx": dx.to(s["x"].dtype), "dgate": s["alpha"] * s["w_post"] * both,
            "dw_post": s["alpha"] * s["gate"] * both, "dw_pre": (dh * n).sum(dim=0)}


def _run_plain(s):
    op = s["op"]
    if op == "fake_quantize":
        return _plain_quantize(s["x"].t() if s["trans"] else s["x"])
    if op == "product_mx4":
        return torch.matmul(_decode(s["a"], s["sa"], s["K"]), _decode(s["b"], s["sb"], s["K"]).t())
    if op == "product_16":
        return torch.matmul(s["a"].float(), _decode(s["b"], s["sb"], s["K"]).t())
    if op == "norm":
        xo, h = _plain_norm(s)
        return {"xo": xo, "h": h}
    return _plain_norm_grad(s)


# ---- the package's calls -------------------------------------------------------

def _run_own(s):
    import linear_layer_amd as ll
    op = s["op"]
    if op == "fake_quantize":
        ll.mx4_quantize(s["x"], s["codes"], s["scales"], trans=s["trans"])
        return ll.mx4_dequantize(s["codes"], s["scales"], s["out"])
    if op == "product_mx4":
        return ll.gemm_mx4f32_nt(s["a"], s["sa"], s["b"], s["sb"], s["out"], K=s["K"])
    if op == "product_16":
        call = ll.gemm_f16mx4f32_nt if s["type"] == "f16" else ll.gemm_bf16mx4f32_nt
        return call(s["a"], s["b"], s["sb"], s["out"])
    if op == "norm":
        ll.rmsnorm_residual(s["y"], s["w_post"], s["gate"], s["alpha"], s["x"], s["w_pre"], s["xo"], s["h"], eps=EPS)
        return {"xo": s["xo"], "h": s["h"]}
    ll.rmsnorm_residual_grad(s["dxo"], s["dh"], s["y"], s["w_post"], s["gate"], s["alpha"], s["x"], s["w_pre"],
                             s["dy"], s["dx"], s["dgate"], s["dw_post"], s["dw_pre"], s["work"], eps=EPS)
    return {k: s[k] for k in ("dy", "dx", "dgate", "dw_post", "dw_pre")}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op, M = case["op"], case["M"]
    if op == "fake_quantize":
        r, c = (case["K"], M) if case["trans"] else (M, case["K"])
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": 2 * size * r * c + r * ((c + 1) // 2 + -(-c // BLOCK)), "flops": 3 * r * c}
    if op in ("product_mx4", "product_16"):
        N, K = case["N"], case["K"]
        row = (K + 1) // 2 + -(-K // BLOCK)
        return {"bytes": N * row + M * (row if op == "product_mx4" else 2 * K) + 4 * M * N, "flops": 2 * M * N * K}
    N, size = case["N"], 4 if case["type"] == "f32" else 2
    if op == "norm":
        return {"bytes": M * N * (4 + 3 * size) + 12 * N, "flops": 10 * M * N}
    return {"bytes": M * N * (8 + 4 * size) + 24 * N, "flops": 25 * M * N}


# ---- from the definitions, in 64 bits -----------------------------------------------

def _exact_values(codes, scales, K):
    """sign * (mantissa scaled by the exponent field) * 2^(scale - 127)."""
    n = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        ex, m = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex - 1))
        n[:, half::2] = torch.where(c >= 8, -mag, mag)
    n = n[:, :K]
    pos = torch.arange(K, device=DEV) // BLOCK
    return n * torch.exp2(scales.double() - 127)[:, pos]


def _exact_quantize(x):
    rows, cols = x.shape
    full = torch.nn.functional.pad(x.double(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = full.abs().amax(dim=2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # log2 rounds next to a power of two: settle it by comparing
    e = e - (torch.exp2(e) > top).double() * (top > 0) + (torch.exp2(e + 1) <= top).double()
    scale = torch.exp2((e - 2).clamp(-127, 127))
    a = full.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0) * scale
    return (q * torch.sign(full)).view(rows, -1)[:, :cols].contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fake_quantize":
        return _exact_quantize(s["x"].t() if case["trans"] else s["x"])
    if op in ("product_mx4", "product_16"):
        K = case["K"]
        a = _exact_values(s["a"], s["sa"], K) if op == "product_mx4" else s["a"].double()
        return a @ _exact_values(s["b"], s["sb"], K).t().contiguous()
    d = {k: s[k].double() for k in ("x", "y", "w_post", "w_pre", "gate")}
    alpha, N = s["alpha"], case["N"]
    ry = 1 / torch.sqrt((d["y"] * d["y"]).sum(1, keepdim=True) / N + EPS)
    xo = d["x"] + alpha * d["gate"] * d["w_post"] * d["y"] * ry
    rx = 1 / torch.sqrt((xo * xo).sum(1, keepdim=True) / N + EPS)
    if op == "norm":
        return {"xo": xo, "h": xo * rx * d["w_pre"]}
    # each output's derivative, written out from r = (sum v^2 / N + eps)^(-1/2): dr/dv = -v r^3 / N
    dxo, dh = s["dxo"].double(), s["dh"].double()
    k = dh * d["w_pre"]
    total = dxo + k * rx - xo * rx ** 3 * ((k * xo).sum(1, keepdim=True) / N)
    c = total * alpha * d["gate"] * d["w_post"]
    dy = c * ry - d["y"] * ry ** 3 * ((c * d["y"]).sum(1, keepdim=True) / N)
    return {"dy": dy, "dx": total, "dgate": (total * alpha * d["w_post"] * d["y"] * ry).sum(0),
            "dw_post": (total * alpha * d["gate"] * d["y"] * ry).sum(0), "dw_pre": (dh * xo * rx).sum(0)}


