"""The example that runs the 4-bit products and the residual norms together: its
results follow FP32 with unpacked weights to 4-bit precision, and a decode step
replayed from a graph follows the prompt's own.

Tolerances. A 4-bit value is off by at most a third of itself or a twelfth of its
block's largest (values past 6 steps are cut to 6 from below 8, others move by at
most half a step): a product of such operands stays within half of its size, and
the residual stream, of which the block is a part, nearer. A decode step differs
from the same row of a prompt by the order of FP32 sums and by 16-bit roundings that
this turns: 2^-8 of a value, through two layers and two norms less than 2^-5."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "low_precision_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("low_precision_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("width,hidden,tokens", [(512, 1376, 33), (1024, 2752, 130), (96, 200, 5)])
def test_example(example, width, hidden, tokens):
    r = example.main(width, hidden, tokens)
    assert r["x"] < 0.5 and r["h"] < 0.5 and r["da"] < 0.5 and r["dw2"] < 0.5
    assert r["decode"] < 2.0 ** -5


def test_decode_graph_follows_new_inputs(example):
    """Replays between the program's own calls equal the eager step bit for bit."""
    block = example.Block(512, 1376)
    step = block.decoder(2)
    for k in range(4):
        x, h = (torch.randn((2, 512), device="cuda").bfloat16() for _ in range(2))
        want = [t.clone() for t in block.forward(x, h)]
        got = step(x, h)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
