"""The attention-block example at small sizes: the operators together, as a user runs them."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(hidden=256, heads=4, kv_heads=2, head_dim=64, requests=3, prompt=90, steps=40),
                                dict(hidden=512, heads=6, kv_heads=1, head_dim=128, requests=8, prompt=300, steps=3),
                                dict(hidden=512, heads=2, kv_heads=2, head_dim=256, requests=1, prompt=1, steps=70)])
def test_attention_block(kw):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    prompt_error, decode_error, us, block = m.run(**kw)
    # bfloat16: keys, values and probabilities at 2^-11 of themselves, the result at 2^-9; float32: a few hundred 2^-24
    assert prompt_error <= 2.0 ** -7
    assert decode_error <= 2e-5
    want = [max(1, kw["prompt"] - 37 * b) + 1 + kw["steps"] for b in range(kw["requests"])]
    assert np.array_equal(block.cached.cpu().numpy(), want)
    used = block.table.cpu().numpy()
    per = [-(-n // block.page) for n in want]
    pages = np.concatenate([used[b, :n] for b, n in enumerate(per)])
    assert (pages >= 0).all() and len(set(pages.tolist())) == len(pages)     # no page serves two requests
