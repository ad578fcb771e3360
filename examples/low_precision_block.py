"""A feed-forward block with its weights in 4 bits: a prompt, decode steps and a
training step, on the operators as a user calls them.

    python examples/low_precision_block.py [--width 4096] [--hidden 11008] [--tokens 2047]

The block is y = relu(h W1^T) W2^T with W1 (hidden x width) and W2 (width x hidden) in
microscaled 4-bit floating point and bfloat16 activations. Between two blocks stands
the residual step x' = x + alpha * gate * rms(y) * w_post, h' = rms(x') * w_pre.

* ``Block.forward`` takes any number of tokens (one: a decode step).
* ``Block.decoder`` captures a decode step into a graph and returns what replays it.
* ``Block.backward`` is the training step's way back: the gradient of the residual
  step, then the second layer's products with both operands in 4 bits, each
  quantised along the axis that its product contracts.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import linear_layer_amd as ll  # noqa: E402


def pack(t, trans=False):
    """(codes, scales) of t's rows, or of its columns as the transposed matrix's rows."""
    rows, n = (t.shape[1], t.shape[0]) if trans else t.shape
    codes, scales = (torch.empty(s, dtype=torch.uint8, device=t.device) for s in ll.mx4_shapes(rows, n))
    return ll.mx4_quantize(t, codes, scales, trans=trans)


class Block:
    def __init__(self, width, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.width, self.hidden, self.device = width, hidden, device
        # the training program's weights; the serving ones are their packed forms
        self.w1 = torch.randn((hidden, width), generator=g, device=device) / width ** 0.5
        self.w2 = torch.randn((width, hidden), generator=g, device=device) / hidden ** 0.5
        self.q1, self.q2 = pack(self.w1), pack(self.w2)
        self.gate, self.w_post, self.w_pre = (1 + 0.1 * torch.randn((width,), generator=g, device=device) for _ in range(3))
        self.alpha = 0.7

    def buffers(self, M):
        """What a forward pass over M tokens writes."""
        bf = dict(dtype=torch.bfloat16, device=self.device)
        return {"up": torch.empty((M, self.hidden), device=self.device), "a": torch.empty((M, self.hidden), **bf),
                "y": torch.empty((M, self.width), device=self.device), "x": torch.empty((M, self.width), **bf),
                "h": torch.empty((M, self.width), **bf)}

    def forward(self, x, h, out=None):
        """(x', h') of the residual stream x and the block's input h (bfloat16, M x width)."""
        b = self.buffers(x.shape[0]) if out is None else out
        ll.gemm_bf16mx4f32_nt(h, *self.q1, b["up"])
        b["a"].copy_(b["up"].relu_())
        ll.gemm_bf16mx4f32_nt(b["a"], *self.q2, b["y"])
        ll.rmsnorm_residual(b["y"], self.w_post, self.gate, self.alpha, x, self.w_pre, b["x"], b["h"])
        return b["x"], b["h"]

    def decoder(self, M=1):
        """step(x, h) -> (x', h') for M tokens at a time, replayed from a graph; the
        result stays in the same two tensors."""
        x, h = (torch.zeros((M, self.width), dtype=torch.bfloat16, device=self.device) for _ in range(2))
        out = self.buffers(M)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x, h, out)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.forward(x, h, out)

        def step(x_new, h_new):
            x.copy_(x_new)
            h.copy_(h_new)
            graph.replay()
            return out["x"], out["h"]
        return step

    def backward(self, dxo, dh, x, saved):
        """The gradients of the residual step and of the second layer: a dict of dx (to
        the residual stream), da (to the layer's input), dw2, dgate, dw_post, dw_pre.
        `saved`: the buffers of the forward pass over x."""
        M, y, a = x.shape[0], saved["y"], saved["a"]
        d = {"dy": torch.empty_like(y), "dx": torch.empty_like(x)}
        for k in ("dgate", "dw_post", "dw_pre"):
            d[k] = torch.empty((self.width,), device=self.device)
        work = torch.empty((ll.rmsnorm_grad_workspace_size(M, self.width),), dtype=torch.uint8, device=self.device)
        ll.rmsnorm_residual_grad(dxo, dh, y, self.w_post, self.gate, self.alpha, x, self.w_pre, d["dy"], d["dx"],
                                 d["dgate"], d["dw_post"], d["dw_pre"], work)
        # da = dy W2 contracts over the width, dw2 = dy^T a over the tokens
        d["da"] = ll.gemm_mx4f32_nt(*pack(d["dy"]), *pack(self.w2, trans=True),
                                    torch.empty((M, self.hidden), device=self.device), K=self.width)
        d["dw2"] = ll.gemm_mx4f32_nt(*pack(d["dy"], trans=True), *pack(a, trans=True),
                                     torch.empty((self.width, self.hidden), device=self.device), K=M)
        return d


def distance(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def reference(block, x, h):
    """The block in FP32 with its unpacked weights: how far 4 bits are from it."""
    y = torch.relu(h.float() @ block.w1.t()) @ block.w2.t()
    rms = lambda v: v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5)  # noqa: E731
    xo = x.float() + block.alpha * block.gate * rms(y) * block.w_post
    return xo, rms(xo) * block.w_pre


def timed(f, n=20):
    f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


def main(width=4096, hidden=11008, tokens=2047):
    block = Block(width, hidden)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, h, dxo, dh = (torch.randn((tokens, width), generator=g, device="cuda").bfloat16() for _ in range(4))
    saved = block.buffers(tokens)
    xo, ho = block.forward(x, h, saved)
    result = dict(zip(("x", "h"), (distance(a, b) for a, b in zip((xo, ho), reference(block, x, h)))))
    step = block.decoder()
    one = step(x[:1], h[:1])
    result["decode"] = distance(one[1], ho[:1])
    grads = block.backward(dxo, dh, x, saved)
    result["da"] = distance(grads["da"], grads["dy"] @ block.w2)
    result["dw2"] = distance(grads["dw2"], grads["dy"].t() @ saved["a"].float())
    print("relative distance from FP32 with unpacked weights:",
          ", ".join(f"{k} {v:.3f}" for k, v in result.items() if k != "decode"))
    print(f"a decode step from the prompt's own token: {result['decode']:.1e}")
    print(f"prompt of {tokens}: {timed(lambda: block.forward(x, h, saved)):.0f} us; "
          f"decode step: {timed(lambda: step(x[:1], h[:1])):.0f} us; "
          f"way back: {timed(lambda: block.backward(dxo, dh, x, saved)):.0f} us")
    return result


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=11008)
    p.add_argument("--tokens", type=int, default=2047)
    a = p.parse_args()
    main(a.width, a.hidden, a.tokens)
