"""The array form of the cache reference (kv_vector.py) is the plain one."""
import numpy as np
import pytest

import kv_reference as ref
import kv_vector as vec


@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (128, 64, 32), (256, 128, 16)])
def test_decode_and_attend(D, group, page):
    rng = np.random.default_rng(D)
    P, H, Hkv = 7, 6, 2
    cache = rng.integers(0, 256, (P, Hkv, page // 16 * ref.tile_bytes(D, group)), dtype=np.uint8)
    tiles = cache.reshape(P, Hkv, page // 16, -1)
    coef = rng.uniform(-1, 1, (P, Hkv, page // 16, 64 * (D // group))).astype(np.float16)
    tiles[..., 16 * D:] = coef.view(np.uint8).reshape(tiles[..., 16 * D:].shape)
    k, v = vec.decode(cache, D, page, group)
    for slot in range(0, P * page, 5):
        for got, want in zip((k, v), ref.values(cache, slot, D, page, group)):
            assert np.array_equal(got[slot // page, :, slot % page], want)
    lens, fresh = [2 * page + 3, 0, 3, page], [4, 2, 5, 0]
    cu = np.concatenate(([0], np.cumsum(fresh)))
    table = rng.permutation(P)[:4][:, None] * np.ones((1, 3), int)
    table[0] = (1, -1, 4)
    table[2, 0] = P + 2
    q = rng.standard_normal((cu[-1], H, D))
    for window in (0, 1, 7):
        for got, want in zip(vec.attend(q, k, v, table, lens, cu, page, 0.1, window),
                             ref.attend(q, cache, table, lens, cu, page, group, 0.1, window)):
            assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
