"""A dense or an expert layer in 16 bits and its training step as measured work.

Five operators, each through the package's public calls:

* ``linear``: ``linear16_nt``, Y = act(X * W^T + b) + R. X and W in 16 bits, FP32 sums; with
  ``groups`` the rows of X are sorted by expert and each expert has a weight of its own.
  ``keep`` writes Z = X * W^T + b down for the way back: in 16 bits, or in microscaled
  8-bit floating point (blocks of 32 along a row, E4M3 values, one E8M0 scale a block).
* ``grad_act``: ``linear16_grad_act``, dZ = dY * act'(Z) with Z in 16 or in 8 bits, and the
  bias's gradient.
* ``grad_input``: ``linear16_grad_input``, dX = dZ * W.
* ``grad_weight``: ``linear16_grad_weight``, dW = beta * dW + dZ^T * X with X in 16 or in 8 bits.
* ``checkpoint``: ``mx8_quantize`` and ``mx8_dequantize``, a tensor into 8 bits and back.

The dense sizes are those of the package's own workloads: the fully-connected layer
4096 -> 11008 and its way back with 1, 33 and 2047 rows. The experts' are generic: 16 of
2048 -> 4096 with 64 and 8191 rows.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 32
TOP = 448.0   # the largest E4M3 value


def listed():
    return [
        # one token through a 4096 -> 11008 layer: latency and weight reading
        {"name": "linear_bf16_1x11008x4096", "op": "linear", "M": 1, "N": 11008, "K": 4096, "groups": 0, "type": "bf16",
         "out": "bf16", "act": "silu", "bias": True, "residual": False, "keep": "", "pad": 0},
        # a training step's ragged batch through the same layer, Z kept in 8 bits
        {"name": "linear_bf16_2047x11008x4096", "op": "linear", "M": 2047, "N": 11008, "K": 4096, "groups": 0,
         "type": "bf16", "out": "bf16", "act": "gelu", "bias": True, "residual": False, "keep": "mx8", "pad": 0},
        # a decode step of 64 tokens over 16 experts: every expert's weight is read for a few rows
        {"name": "experts_bf16_64x4096x2048", "op": "linear", "M": 64, "N": 4096, "K": 2048, "groups": 16, "type": "bf16",
         "out": "bf16", "act": "silu", "bias": False, "residual": False, "keep": "", "pad": 0},
        # a prompt's tokens through the experts' way back to the residual stream in FP32
        {"name": "experts_bf16_8191x2048x4096", "op": "linear", "M": 8191, "N": 2048, "K": 4096, "groups": 16,
         "type": "bf16", "out": "f32", "act": "none", "bias": True, "residual": True, "keep": "", "pad": 0},
        # the activation's gradient of a training step over experts, Z read from 8 bits
        {"name": "gradact_bf16_8191x4096", "op": "grad_act", "M": 8191, "N": 4096, "groups": 16, "type": "bf16", "out": "bf16",
         "act": "silu", "keep": "mx8", "bias": True, "pad": 0},
        # a small odd one, rows off a vector's alignment
        {"name": "gradact_f16_129x1001", "op": "grad_act", "M": 129, "N": 1001, "groups": 0, "type": "f16", "out": "f32",
         "act": "gelu_tanh", "keep": "z16", "bias": True, "pad": 0},
        # the gradient that leaves the experts' first layer
        {"name": "gradinput_bf16_8191x4096x2048", "op": "grad_input", "M": 8191, "N": 4096, "K": 2048, "groups": 16,
         "type": "bf16", "out": "bf16", "pad": 0},
        # the way back through the dense layer for a short ragged batch in binary16
        {"name": "gradinput_f16_2047x11008x4096", "op": "grad_input", "M": 2047, "N": 11008, "K": 4096, "groups": 0,
         "type": "f16", "out": "f16", "pad": 0},
        # the dense weight's gradient from inputs kept in 8 bits, added to the one before it in FP32
        {"name": "gradweight_bf16_2047x11008x4096", "op": "grad_weight", "M": 2047, "N": 11008, "K": 4096, "groups": 0,
         "type": "bf16", "out": "f32", "beta": 1.0, "keep": "mx8", "pad": 0},
        # the experts' weights' gradients
        {"name": "gradweight_bf16_8191x4096x2048", "op": "grad_weight", "M": 8191, "N": 4096, "K": 2048, "groups": 16,
         "type": "bf16", "out": "bf16", "beta": 0.0, "keep": "", "pad": 0},
        # the inputs of a long batch put into 8 bits for the way back, and read again
        {"name": "checkpoint_bf16_8192x8192", "op": "checkpoint", "M": 8192, "K": 8192, "type": "bf16", "pad": 0},
        # those of a few rows: latency
        {"name": "checkpoint_f32_4x4096", "op": "checkpoint", "M": 4, "K": 4096, "type": "f32", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "grad_act", "grad_input", "grad_weight", "grad_weight", "checkpoint"])
    pad, t = rng.choice([0, 0, 0, 1, 8]), rng.choice(["f16", "bf16"])
    if op == "checkpoint":
        M, K = _log(rng, 1, 8192), _log(rng, 32, 11008)
        return {"op": op, "M": min(M, 8192 * 8192 // K), "K": K, "type": rng.choice(list(TYPES)), "pad": pad}
    groups = rng.choice([0, 0, 4, 16, 64])
    M, N = _log(rng, 1, 8192), _log(rng, 64, 11008)
    c = {"op": op, "M": M, "N": N, "groups": groups, "type": t, "out": rng.choice([t, t, "f32"]), "pad": pad}
    if op == "grad_act":
        return {**c, "act": rng.choice(ACTS), "keep": rng.choice(["z16", "mx8"]), "bias": rng.random() < 0.7}
    K = _log(rng, 64, 11008)
    if rng.random() < 0.7:   # whole vectors, as models have them
        N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
    # the product, and all experts' weights, within the largest listed cases'
    N = max(1, min(N, 2047 * 11008 * 4096 // (2 * M * K), (1 << (26 if c["out"] == "f32" else 27)) // (max(groups, 1) * K)))
    c |= {"N": N, "K": K}
    if op == "linear":
        return {**c, "act": rng.choice(ACTS), "bias": rng.random() < 0.7, "residual": rng.random() < 0.4,
                "keep": rng.choice(["", "", "z16", "mx8"])}
    if op == "grad_weight":
        c |= {"beta": rng.choice([0.0, 1.0]), "keep": rng.choice(["", "mx8"])}
    return c


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _rows(rows, cols, pad, dtype):
    """rows x cols whose rows lie cols + pad elements apart."""
    return torch.zeros((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _activations(g, rows, cols, dtype, pad, scale=1.0):
    """Normal values with channels of different size, as hidden states have them."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= scale * torch.exp(0.5 * torch.randn((cols,), generator=g, device=DEV))
    out = _rows(rows, cols, pad, dtype)
    out.copy_(x)
    return out


def _live(M, groups):
    """How many of the experts get rows: an eighth of them has none."""
    return min(M, groups - groups // 8)


def _route(seed, M, groups):
    """Rows of each expert: some have none, the others very different numbers."""
    g = torch.Generator()
    g.manual_seed(seed * 104729 + 11)
    live = _live(M, groups)
    share = torch.exp(0.6 * torch.randn((live,), generator=g, dtype=torch.float64))
    ends = torch.round(torch.cumsum(share, 0) / share.sum() * (M - live)).long()
    n = torch.diff(ends, prepend=torch.zeros(1, dtype=torch.long)) + 1
    counts = torch.zeros(groups, dtype=torch.long)
    counts[torch.randperm(groups, generator=g)[:live]] = n
    return counts


def _weights(g, groups, N, K, pad, dtype):
    """One weight N x K, or a stack of them with a 0th axis."""
    w = torch.zeros((max(groups, 1), N, K + pad), dtype=dtype, device=DEV)[:, :, :K]
    for i in range(w.shape[0]):
        w[i] = torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)
    return w if groups else w[0]


def _kept(x, pad):
    """x in 8 bits, as an earlier step's forward pass wrote it down: codes and scales."""
    rows, K = x.shape
    v, e = _scaled(x.float())
    codes, scales = _rows(rows, K, pad, torch.uint8), _rows(rows, v.shape[1], pad, torch.uint8)
    codes.copy_(v.reshape(rows, -1)[:, :K].contiguous().to(torch.float8_e4m3fn).view(torch.uint8))
    scales.copy_((e[:, :, 0] + 127).to(torch.uint8))
    return codes, scales


def prepare(case, seed):
    g, pad, op, M = _gen(seed), case["pad"], case["op"], case["M"]
    s = dict(case)
    t = TYPES[case["type"]]
    if op == "checkpoint":
        K = case["K"]
        s["x"] = _activations(g, M, K, t, pad)
        s["codes"], s["scales"] = _rows(M, K, pad, torch.uint8), _rows(M, -(-K // BLOCK), pad, torch.uint8)
        s["y"] = torch.empty((M, K), dtype=t, device=DEV)
        return s
    N, groups, out = case["N"], case["groups"], TYPES[case["out"]]
    s["offsets"] = None
    if groups:
        counts = _route(seed, M, groups)
        s["most"] = int(counts.max())
        s["offsets"] = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32).to(DEV)
    if op == "linear":
        K = case["K"]
        s["x"], s["w"] = _activations(g, M, K, t, pad), _weights(g, groups, N, K, pad, t)
        s["b"] = 0.2 * torch.randn((max(groups, 1), N), generator=g, device=DEV) if case["bias"] else None
        if s["b"] is not None and not groups:
            s["b"] = s["b"][0]
        s["r"] = _activations(g, M, N, out, pad) if case["residual"] else None
        s["y"] = _rows(M, N, pad, out)
        if case["keep"] == "z16":
            s["z"] = _rows(M, N, pad, t)
        elif case["keep"] == "mx8":
            s["z"] = _rows(M, N, pad, torch.uint8), _rows(M, -(-N // BLOCK), pad, torch.uint8)
            s["z_values"] = torch.empty((M, N), dtype=t, device=DEV)
    elif op == "grad_act":
        s["dy"] = _activations(g, M, N, out, pad, 0.1)
        z = _activations(g, M, N, t, pad)
        s["z"] = z if case["keep"] == "z16" else _kept(z, pad)
        s["dz"] = _rows(M, N, pad, t)
        s["db"] = torch.empty((groups, N) if groups else (N,), device=DEV) if case["bias"] else None
    else:
        K = case["K"]
        s["dz"] = _activations(g, M, N, t, pad, 0.1)
        if op == "grad_input":
            s["w"], s["dx"] = _weights(g, groups, N, K, pad, t), _rows(M, K, pad, out)
        else:
            x = _activations(g, M, K, t, pad)
            s["x"] = _kept(x, pad) if case["keep"] == "mx8" else x
            shape = (groups, N, K) if groups else (N, K)
            # with beta, what the passes so far have summed up; every pass adds to it
            s["dw"] = (0.5 * torch.randn(shape, generator=g, device=DEV)).to(out)
    return s


# ---- the plain forms ----------------------------------------------------------

def _blocks(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.zeros((rows, nb * BLOCK), device=DEV)
    v[:, :cols] = x
    return v.view(rows, nb, BLOCK)


def _scaled(x):
    """x's blocks over their scales 2^e, and e: the smallest with which the block's largest is at most 448."""
    v = _blocks(x)
    m, e = torch.frexp(v.abs().amax(dim=2, keepdim=True))   # top = m * 2^e, m in [0.5, 1)
    e = e - 9 + (m > TOP / 512).int()
    e = torch.where(m == 0, -127, e.clamp(-127, 127))
    return torch.ldexp(v, -e), e


def _round8(v):
    """v rounded to E4M3: 3 fraction bits, none below 2^-9; ties to even."""
    e = (torch.frexp(v).exponent - 1).clamp(min=-6) - 3
    return torch.ldexp(torch.round(torch.ldexp(v, -e)), e)


def _through8(x, dtype):
    """x as 8 bits hold it."""
    v, e = _scaled(x)
    return torch.ldexp(_round8(v), e).reshape(x.shape[0], -1)[:, :x.shape[1]].to(dtype).contiguous()


def _decode(codes, scales):
    """The values that codes and scales stand for, in 32 bits."""
    i = torch.arange(256, device=DEV)
    ex, frac = (i >> 3) & 15, (i & 7).float()
    table = torch.where(ex == 0, torch.ldexp(frac, torch.full_like(ex, -9)), torch.ldexp(8 + frac, ex - 10))
    table = torch.where(i >= 128, -table, table)
    e = torch.repeat_interleave(scales.int() - 127, BLOCK, dim=1)[:, :codes.shape[1]]
    return torch.ldexp(table[codes.long()], e)


def _value(v):
    return _decode(*v) if isinstance(v, tuple) else v.float()


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _by_group(s):
    """Row numbers, group by group, each padded to the longest; which of them are rows; and
    the group and place of each row."""
    off, M = s["offsets"].long(), s["M"]
    at = off[:-1, None] + torch.arange(s["most"], device=DEV)
    row = torch.arange(M, device=DEV)
    group = torch.searchsorted(off[1:], row, right=True)
    return at.clamp(max=M - 1), (at < off[1:, None])[:, :, None], (group, row - off[group])


def _plain_linear(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"]
    if s["groups"]:
        at, _, back = _by_group(s)
        z = torch.matmul(x[at], w.transpose(1, 2))[back]
        if b is not None:
            z = z + b[back[0]]
    else:
        z = torch.matmul(x, w.t())
        if b is not None:
            z = z + b
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(s["y"].dtype)}
    if s["keep"]:
        t = TYPES[s["type"]]
        out["z"] = _through8(z, t) if s["keep"] == "mx8" else z.to(t)
    return out


def _plain_grad_act(s):
    dz = s["dy"].float() * _act_slope(_value(s["z"]), s["act"])
    out = {"dz": dz.to(s["dz"].dtype)}
    if s["db"] is not None:
        if s["groups"]:
            at, real, _ = _by_group(s)
            out["db"] = (dz[at] * real).sum(dim=1)
        else:
            out["db"] = dz.sum(dim=0)
    return out


def _plain_grad_input(s):
    dz, w = s["dz"].float(), s["w"].float()
    if s["groups"]:
        at, _, back = _by_group(s)
        return torch.matmul(dz[at], w)[back].to(s["dx"].dtype)
    return torch.matmul(dz, w).to(s["dx"].dtype)


def _plain_grad_weight(s):
    dz, x = s["dz"].float(), _value(s["x"])
    if s["groups"]:
        at, real, _ = _by_group(s)
        dw = torch.matmul((dz[at] * real).transpose(1, 2), x[at])
    else:
        dw = torch.matmul(dz.t(), x)
    if s["beta"]:
        dw = dw + s["beta"] * s["dw"].float()
    return s["dw"].copy_(dw)


def _run_plain(s):
    op = s["op"]
    if op == "linear":
        return _plain_linear(s)
    if op == "grad_act":
        return _plain_grad_act(s)
    if op == "grad_input":
        return _plain_grad_input(s)
    if op == "grad_weight":
        return _plain_grad_weight(s)
    return _through8(s["x"].float(), s["x"].dtype)


# ---- the package's calls -------------------------------------------------------

def _run_own(s):
    import linear_layer_amd as ll
    op = s["op"]
    if op == "checkpoint":
        ll.mx8_quantize(s["x"], s["codes"], s["scales"])
        return ll.mx8_dequantize(s["codes"], s["scales"], s["y"])
    if op == "linear":
        act = getattr(ll, "ACT_" + s["act"].upper())
        ll.linear16_nt(s["x"], s["w"], s["b"], act, s["r"], s["y"], Z=s.get("z"), offsets=s["offsets"])
        out = {"y": s["y"]}
        if s["keep"] == "mx8":   # as the values that its 8 bits stand for
            out["z"] = ll.mx8_dequantize(*s["z"], s["z_values"])
        elif s["keep"]:
            out["z"] = s["z"]
        return out
    if op == "grad_act":
        act = getattr(ll, "ACT_" + s["act"].upper())
        ll.linear16_grad_act(s["dy"], s["z"], act, s["dz"], s["db"], offsets=s["offsets"])
        return {"dz": s["dz"]} if s["db"] is None else {"dz": s["dz"], "db": s["db"]}
    if op == "grad_input":
        return ll.linear16_grad_input(s["dz"], s["w"], s["dx"], offsets=s["offsets"])
    return ll.linear16_grad_weight(s["dz"], s["x"], s["dw"], beta=s["beta"], offsets=s["offsets"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op, M = case["op"], case["M"]
    size = {"f32": 4, "f16": 2, "bf16": 2, "z16": 2, "": 2}

    def held(rows, cols, how):
        return rows * (cols + -(-cols // BLOCK)) if how == "mx8" else rows * cols * size[how]

    if op == "checkpoint":
        K = case["K"]
        return {"bytes": 2 * size[case["type"]] * M * K + held(M, K, "mx8"), "flops": 3 * M * K}
    N, groups, out = case["N"], case["groups"], size[case["out"]]
    if op == "grad_act":
        bytes = M * N * (out + 2) + (held(M, N, case["keep"]) if case["act"] != "none" else 0)
        return {"bytes": bytes + (4 * max(groups, 1) * N if case["bias"] else 0), "flops": 10 * M * N}
    K, live = case["K"], _live(M, groups) if groups else 1
    flops = 2 * M * N * K
    if op == "linear":
        bytes = 2 * M * K + 2 * live * N * K + M * N * out * (2 if case["residual"] else 1)
        return {"bytes": bytes + (held(M, N, case["keep"]) if case["keep"] else 0) + (4 * live * N if case["bias"] else 0),
                "flops": flops}
    if op == "grad_input":
        return {"bytes": 2 * M * N + 2 * live * N * K + M * K * out, "flops": flops}
    return {"bytes": 2 * M * N + held(M, K, case["keep"]) + max(groups, 1) * N * K * out * (2 if case["beta"] else 1),
            "flops": flops}


# ---- from the definitions, in 64 bits -----------------------------------------------

def _exact8(x):
    rows, cols = x.shape
    full = torch.nn.functional.pad(x.double(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = full.abs().amax(dim=2, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / TOP))
    # the logarithm rounds next to a border: settle it by comparing
    e = e + (torch.exp2(e) * TOP < top).double() - (torch.exp2(e - 1) * TOP >= top).double()
    scale = torch.exp2(torch.where(top > 0, e, -127.0).clamp(-127, 127))
    a = full.abs() / scale
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    step = torch.where(a >= 16 * step, 2 * step, step)
    return (torch.round(a / step) * step * scale * torch.sign(full)).view(rows, -1)[:, :cols].contiguous()


def _exact_value(v):
    if not isinstance(v, tuple):
        return v.double()
    codes, scales = v
    c = codes.long()
    ex, f = ((c >> 3) & 15).double(), (c & 7).double() / 8
    mag = torch.where(ex == 0, f * 2.0 ** -6, (1 + f) * torch.exp2(ex - 7))
    pos = torch.arange(codes.shape[1], device=DEV) // BLOCK
    return torch.where(c >= 128, -mag, mag) * torch.exp2(scales.double() - 127)[:, pos]


def _exact_act(z, act):
    """act(z) and its slope."""
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("gelu_tanh", "silu"):
        # z * sigmoid(u): u = z, or twice the tanh's argument
        c = 2 * math.sqrt(2 / math.pi)
        u, du = (z, torch.ones_like(z)) if act == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2))
        p = torch.sigmoid(u)
        return z * p, p + z * p * torch.sigmoid(-u) * du
    return z, torch.ones_like(z)


def _spans(s):
    if not s["groups"]:
        return [(0, s["M"])]
    off = s["offsets"].tolist()
    return list(zip(off[:-1], off[1:]))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return _exact8(s["x"])
    spans, G = _spans(s), bool(case["groups"])
    if op == "linear":
        parts = []
        for i, (a, e) in enumerate(spans):
            z = s["x"][a:e].double() @ (s["w"][i] if G else s["w"]).double().t().contiguous()
            parts.append(z if s["b"] is None else z + (s["b"][i] if G else s["b"]).double())
        z = torch.cat(parts)
        y = _exact_act(z, case["act"])[0]
        out = {"y": y if s["r"] is None else y + s["r"].double()}
        if case["keep"]:
            out["z"] = _exact8(z) if case["keep"] == "mx8" else z
        return out
    if op == "grad_act":
        dz = s["dy"].double() * _exact_act(_exact_value(s["z"]), case["act"])[1]
        out = {"dz": dz}
        if s["db"] is not None:
            db = torch.stack([dz[a:e].sum(0) for a, e in spans])
            out["db"] = db if G else db[0]
        return out
    dz = s["dz"].double()
    if op == "grad_input":
        return torch.cat([dz[a:e] @ (s["w"][i] if G else s["w"]).double() for i, (a, e) in enumerate(spans)])
    x = _exact_value(s["x"])
    dw = torch.stack([dz[a:e].t().contiguous() @ x[a:e] for a, e in spans])
    dw = dw if G else dw[0]
    return dw + case["beta"] * s["dw"].double() if case["beta"] else dw
