"""kv_attend where its teams and persistent CTAs take many items one after the other, against float64 (kv_vector.py)."""
import numpy as np
import pytest

import kv_vector as vec
from test_kv_gpu import dev, make_cache, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build, qmm as q
    build.build()
    return q


def check_items(qmm, rng, lens, fresh, H, Hkv, D, group, page, dtype, window=0, runs=3, change=None):
    """One call, checked against float64, and `runs` more that have to give the same bits.  change(cache, table) may put
    other bytes into the cache; each group of elements then has a bound by its own values."""
    import torch
    B, scale = len(lens), D ** -0.5
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 1
    cache, perm = make_cache(rng, pages, Hkv, D, page, group), rng.permutation(pages).astype(np.int32)
    table, at = np.full((B, max(1, max(per))), -1, np.int32), 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
    if change is not None:
        change(cache, table)
    cu = np.concatenate(([0], np.cumsum(fresh))).astype(np.int32)
    q = dev(rng.standard_normal((int(cu[-1]), H, D)).astype(np.float32)).to(getattr(torch, dtype))
    most = max(1, max(fresh))
    ws = qmm.kv_attend_workspace(B, H, Hkv, D, most)
    args = (q, dev(cache), dev(table), dev(np.array(lens, np.int32)), page, group, ws)
    kw = dict(cu=dev(cu), max_fresh=most, scale=scale, window=window)
    out = qmm.kv_attend(*args, **kw, out=torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"))
    again = [qmm.kv_attend(*args, **kw) for _ in range(runs)]
    qmm.check()
    assert not ws[:4096].any()
    k, v = vec.decode(cache, D, page, group)
    qh, at = q.float().cpu().numpy(), (table, lens, cu, page, scale, window)
    want, sizes = vec.attend(qh, k, v, *at)
    got = out.float().cpu().numpy().astype(np.float64)
    tol = np.broadcast_to(tolerance(sizes, want, max(lens), D, dtype), want.shape).copy()
    if change is not None:
        for g in np.arange(0, D, group):
            part = np.zeros(D)
            part[g:g + group] = 1.0
            tol[..., g:g + group] = tolerance(vec.attend(qh, k, v * part, *at)[1], want, max(lens), D, dtype)[..., g:g + group]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), f"{np.max(np.abs(got - want) / tol):.2f} of the tolerance"
    assert all(torch.equal(out, x) for x in again)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_teams_that_list_many_times(qmm, dtype):
    """A team lists 32 requests, and as many items, at a time: here its run holds several lists, some of them empty."""
    rng = np.random.default_rng(43)
    lens, fresh = rng.integers(0, 50, 3000), rng.integers(1, 3, 3000)
    fresh[200:290], fresh[1000:1064] = 0, 0                # runs of requests that ask nothing
    fresh[2900:] = 0
    check_items(qmm, rng, lens.tolist(), fresh.tolist(), 8, 8, 64, 64, 16, dtype, runs=20)


def takes_tiles(B, H, Hkv, D, most):
    """These cases go to the prompt kernel, which takes tiles of 128 rows, with items for several turns of every SM."""
    import torch
    from quantized_weight_gb300 import qmm
    items = B * Hkv * -(-most * H // Hkv // (128 if D == 256 else 256))
    return items > 2 * torch.cuda.get_device_properties(0).multi_processor_count and \
        qmm.kv_attend_tiles(torch.bfloat16, B, H, Hkv, D, most)


@pytest.mark.parametrize("blocks", [2, 1, 4, 3])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (128, 32), (256, 64)])
def test_items_of_one_tile_before_items_of_two(qmm, D, group, blocks):
    """A persistent CTA's score buffers belong to one row tile in turn or to two side by side, as its items come; here items
    of one tile and two (an even number too) blocks of keys stand between items of two tiles, some of which see nothing."""
    rng = np.random.default_rng(100 * D + blocks)
    KB, H, Hkv, B = 64 if D == 256 else 128, 32, 8, 80
    fresh = [20 if b % 2 else 64 for b in range(B)]        # 80 rows or 256
    lens = [int(rng.integers(max(KB * (blocks - 1), 20) + 1, KB * blocks + 1)) if b % 2 else int(rng.integers(64, 3 * KB))
            for b in range(B)]
    fresh[7], lens[10], lens[33] = 0, 0, 9
    assert takes_tiles(B, H, Hkv, D, 64)
    check_items(qmm, rng, lens, fresh, H, Hkv, D, group, 32, "bfloat16", runs=8)


@pytest.mark.parametrize("window", [0, 1, 130])
@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (128, 128, 64), (256, 64, 32)])
def test_items_of_ragged_steps(qmm, D, group, page, window):
    """Single tokens, drafts, chunks and empty requests in one step."""
    rng = np.random.default_rng(D + window)
    B, H, Hkv = 70, 32, 8
    fresh = rng.choice([0, 1, 1, 1, 4, 17, 33, 70, 150], B)
    fresh[0] = 150
    lens = np.maximum(0, fresh + rng.integers(-4, 700, B))
    assert takes_tiles(B, H, Hkv, D, 150)
    check_items(qmm, rng, lens.tolist(), fresh.tolist(), H, Hkv, D, group, page, "bfloat16", window=window, runs=5)
