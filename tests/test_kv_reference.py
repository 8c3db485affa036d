"""The cache reference the GPU tests compare with, pinned on its own: the layout is a bijection onto the tile's code
nibbles, writes read back, the step plan by hand, attention in closed forms."""
import numpy as np
import pytest

import kv_reference as ref


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_is_a_bijection(D):
    kb, kn, vb, vn = ref.places(D)
    k, v = set(zip(kb.ravel(), kn.ravel())), set(zip(vb.ravel(), vn.ravel()))
    assert len(k) == len(v) == 16 * D
    assert {b for b, _ in k} == set(range(8 * D)) and {b for b, _ in v} == set(range(8 * D, 16 * D))
    # a byte of either area belongs to one token, so appending one never touches another's codes
    for by in (kb, vb):
        owner = {}
        for j in range(16):
            for x in by[j]:
                assert owner.setdefault(int(x), j) == j


@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (128, 64, 64), (256, 128, 32)])
def test_put_get(D, group, page):
    rng = np.random.default_rng(D)
    cache = rng.integers(0, 256, (3, 2, page // 16 * ref.tile_bytes(D, group)), dtype=np.uint8)
    G = D // group
    rows = {}
    for slot in (0, 5, page - 1, page + 3, 2 * page + page // 2):
        for h in range(2):
            rows[slot, h] = [(rng.integers(0, 16, D), rng.random(G).astype(np.float16), rng.random(G).astype(np.float16))
                             for _ in range(2)]
            ref.put(cache, slot, h, *rows[slot, h], D, page, group)
    for (slot, h), want in rows.items():
        for a, b in zip(ref.get(cache, slot, h, D, page, group), want):
            assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_plan_by_hand():
    table = np.full((3, 4), -7, np.int32)
    table[0, 0], table[2, :2] = 9, (4, 5)
    t, slots, pos, cu, lens, need = ref.plan([15, 0, 32], [3, 0, 1], [1, 2, 3], table, 6, 16)
    assert t.tolist() == [[9, 1, -7, -7], [-7] * 4, [4, 5, 2, -7]]
    assert slots.tolist() == [9 * 16 + 15, 16, 17, 32, -1, -1] and pos.tolist() == [15, 16, 17, 32, 0, 0]
    assert cu.tolist() == [0, 3, 3, 4] and lens.tolist() == [18, 0, 33] and need.tolist() == [2]


def test_attend_closed_forms():
    D, group, page = 64, 64, 16
    rng = np.random.default_rng(1)
    cache = np.zeros((2, 1, ref.tile_bytes(D, group)), np.uint8)
    for slot in range(32):
        zero = (np.zeros(D, int), np.zeros(1), np.zeros(1))
        ref.put(cache, slot, 0, zero, (np.full(D, slot % 16), np.ones(1), np.zeros(1)), D, page, group)
    q = rng.standard_normal((3, 2, D))
    table = np.array([[1, 0]], np.int32)
    # equal scores: the mean over what is seen; positions 2, 3, 4 of 5 tokens
    out, _ = ref.attend(q, cache, table, [5], [0, 3], page, group, 1.0, 0)
    assert np.allclose(out[:, :, 0], [[1.0] * 2, [1.5] * 2, [2.0] * 2])
    out, _ = ref.attend(q, cache, table, [5], [0, 3], page, group, 1.0, 2)
    assert np.allclose(out[:, :, 0], [[1.5] * 2, [2.5] * 2, [3.5] * 2])
    out, _ = ref.attend(q, cache, table, [2], [0, 3], page, group, 1.0, 0)      # the first query stands before the start
    assert np.allclose(out[:, :, 0], [[0.0] * 2, [0.0] * 2, [0.5] * 2])
