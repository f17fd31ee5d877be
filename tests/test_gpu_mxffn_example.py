"""The example of the gated block: it runs, and its gradients are those of the block in float32 up to what
4-bit operands and 8-bit checkpoints leave."""
import importlib.util
import os

import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("mxfp4_ffn", os.path.join(ROOT, "examples", "mxfp4_ffn.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(example):
    lines = []
    losses, few, many = example.main(steps=3, tokens=300, width=160, hidden=224, log=lines.append)
    assert len(losses) == 3 and all(map(lambda v: v == v and v < float("inf"), losses))
    assert len(lines) == 3      # of the first step, the last, and what was served
    assert few.shape == many.shape == (5, 160) and torch.isfinite(few).all()


def test_gradients_point_the_same_way(example):
    """The cosine to the float32 gradients.  An MXFP4 copy to nearest under the rule that never saturates has a
    relative error of at most half a step in an interval of a factor of 1.5 to 2: uniform over the grid's cells
    (steps 1/2 up to 2, 1 up to 4, 2 up to 6) with amax between 3 and 6 scales, rms(error) <= step / sqrt(12) of about
    0.29 to 0.58 scales at a value rms of a third of amax or more for normal data, 1 to 2 scales: below 0.3.  Stochastic
    rounding doubles the variance: below 0.42.  A product's relative error is at most the root of the sum of its
    operands' squares; with H quantized from such products, and H again in the backward pass, five such errors
    meet at most: sqrt(3 * 0.3^2 + 2 * 0.42^2) = 0.79 and a cosine of 1 / sqrt(1 + 0.79^2) = 0.78."""
    gen = torch.Generator(device=dev()).manual_seed(1)
    rand = lambda *s, std=1.0: std * torch.randn(s, generator=gen, device=dev())
    x = rand(512, 256).bfloat16().requires_grad_()
    w1, w2 = rand(768, 256, std=256 ** -0.5).requires_grad_(), rand(256, 384, std=384 ** -0.5).requires_grad_()
    dy = rand(512, 256).bfloat16()
    got = torch.autograd.grad(example.GatedBlock.apply(x, w1, w2, 7), (x, w1, w2), dy)
    xf = x.detach().float().requires_grad_()
    g, u = (xf @ w1.t()).chunk(2, dim=1)
    want = torch.autograd.grad((torch.nn.functional.silu(g) * u) @ w2.t(), (xf, w1, w2), dy.float())
    for a, b, name in zip(got, want, ("dx", "dW1", "dW2")):
        cos = torch.nn.functional.cosine_similarity(a.double().flatten(), b.double().flatten(), dim=0).item()
        print(name, cos, flush=True)
        assert a.shape == b.shape and cos > 0.78, name
