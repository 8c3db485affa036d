"""The expert-layer example at small sizes: the operators together, as a user runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(hidden=256, width=160, experts=12, top=3, tokens=300, step=5, steps=3),
                                dict(hidden=512, width=384, experts=5, top=1, tokens=1000, step=1, steps=2),
                                dict(hidden=1024, width=416, experts=64, top=8, tokens=77, step=32, steps=2)])
def test_expert_layer(kw):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    prompt_error, step_error, prompt_us, step_us = m.run(**kw)
    # h is rounded (bfloat16: 2^-8 of itself; float32: its sums by some 2^-20) and then quantized, so a value next to a border
    # between two codes, a step of a quarter or more of itself apart, may go the other way: with a probability of the error over
    # the step, 2^-8 / 2^-2 (2^-20 / 2^-2).  So many of the products' terms differ by a quarter: the square root of their share
    # times a quarter, 2^-5 (2^-11); bfloat16 results add 2^-8.
    assert prompt_error <= 2.0 ** -5 + 2.0 ** -8
    assert step_error <= 2.0 ** -11
    assert prompt_us > 0 and step_us > 0
