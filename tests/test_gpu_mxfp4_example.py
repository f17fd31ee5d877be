"""The example that runs the MXFP4 operators together: it learns, and serves the same result for
a few tokens as for many."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_experts.py")


def test_expert_layer_learns_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("mxfp4_experts", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, few, many = example.main(steps=40, tokens=1024)
    assert losses[-1] < 0.5 * losses[0]
    assert torch.isfinite(few).all()
    # products differ only in the order of FP32 sums; the second layer's input may round to another
    # code where the first layer's bfloat16 output does
    assert (few.float() - many.float()).norm() <= 0.05 * many.float().norm()
