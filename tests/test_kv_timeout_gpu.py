"""A bounded wait of the attention's prompt kernel that runs out, on the GPU, without faulting or hanging it: the test hook makes
a softmax warp of every block wait on a barrier that nothing completes.  All roles of the block have to leave, the launch
to be reported once, its workspace to be ready, and the next call on it to be right."""
import numpy as np
import pytest

import kv_vector as vec
from test_kv_gpu import dev, make_cache, tolerance

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture(scope="module")
def qmm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build, qmm as q
    build.build()
    q.check()                     # start from a clean status
    return q


# one item a block; several, of one row tile and two, with one block of keys and many
@pytest.mark.parametrize("B,most,length", [(1, 140, 150), (80, 64, 100), (80, 20, 700)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wait_runs_out_then_the_next_call_is_normal(qmm, D, B, most, length):
    import torch
    rng = np.random.default_rng(D + B)
    H, Hkv, page, group = (64, 2, 16, 64) if B == 1 else (32, 8, 16, 64)
    blocks = -(-length // page)
    cache = make_cache(rng, B * blocks, Hkv, D, page, group)
    table = rng.permutation(B * blocks).astype(np.int32).reshape(B, blocks)
    lens, cu = [length] * B, np.arange(B + 1, dtype=np.int32) * most
    q = dev(rng.standard_normal((B * most, H, D)).astype(np.float32)).bfloat16()
    ws = qmm.kv_attend_workspace(B, H, Hkv, D, most)
    out = torch.full_like(q, 7.0)
    args = (q, dev(cache), dev(table), dev(np.array(lens, np.int32)), page, group, ws)
    kw = dict(cu=dev(cu), max_fresh=most, out=out)
    torch.cuda.synchronize()
    qmm.test_timeout_next_attend(200_000)
    qmm.kv_attend(*args, **kw)
    with pytest.raises(qmm.QmmError) as e:
        qmm.check()
    assert e.value.status == TIMEOUT
    qmm.check()                   # reported once
    assert bool((out == 7.0).all()) and not ws[:4096].any()
    for _ in range(2):            # the hook was taken by one launch only
        qmm.kv_attend(*args, **kw)
    qmm.check()
    want, sizes = vec.attend(q.float().cpu().numpy(), *vec.decode(cache, D, page, group), table, lens, cu, page, D ** -0.5, 0)
    err = np.abs(out.float().cpu().numpy() - want)
    assert (err <= tolerance(sizes, want, length, D, "bfloat16")).all() and not ws[:4096].any()


def test_the_hook_waits_for_the_prompt_kernel(qmm):
    """Calls on the other kernel leave it set; limits out of range are refused."""
    import torch
    for limit in (10, 10 ** 9):
        with pytest.raises(qmm.QmmError):
            qmm.test_timeout_next_attend(limit)
    cache = qmm.kv_cache(12, 2, 64, 16)
    table, lens = torch.arange(10, dtype=torch.int32, device="cuda")[None], dev(np.array([150], np.int32))
    q = torch.randn(140, 64, 64, device="cuda")
    ws, cu = qmm.kv_attend_workspace(1, 64, 2, 64, 140), dev(np.array([0, 140], np.int32))
    qmm.test_timeout_next_attend(200_000)
    qmm.kv_attend(q, cache, table, lens, 16, 64, ws, cu=cu, max_fresh=140)
    qmm.check()
    qmm.kv_attend(q.bfloat16(), cache, table, lens, 16, 64, ws, cu=cu, max_fresh=140)
    with pytest.raises(qmm.QmmError):
        qmm.check()
    qmm.check()
