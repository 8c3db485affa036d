"""Plain, slow reference of the 4-bit key/value cache operators: numpy on the CPU, 64-bit where numbers are computed,
sharing nothing with the library.  The cache layout is restated here from include/qmm.h's and kv_layout.cuh's words,
element by element."""
import numpy as np


def tile_bytes(D, group):
    return 16 * D + 128 * (D // group)


def plan(cached, fresh, free, table, tokens, page):
    """(table, slots, positions, cu, lens, need) of one step."""
    table = table.copy()
    slots, positions = np.full(tokens, -1, np.int32), np.zeros(tokens, np.int32)
    cu, lens, taken, t = [0], [], 0, 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        c, f = max(0, int(c)), max(0, int(f))
        have, tot = -(-c // page), -(-(c + f) // page)
        pages = {}
        for col in range(have, tot):
            pages[col] = int(free[taken]) if taken < len(free) else -1
            taken += 1
            if col < table.shape[1]:
                table[b, col] = pages[col]
        for i in range(f):
            pos = c + i
            col = pos // page
            if t < tokens:
                positions[t] = pos
                pg = -1 if col >= table.shape[1] else int(table[b, col])
                slots[t] = pg * page + pos % page if pg >= 0 else -1
            t += 1
        cu.append(cu[-1] + f)
        lens.append(c + f)
    return table, slots, positions, np.array(cu, np.int32), np.array(lens, np.int32), np.array([taken], np.int32)


def _row(j):
    return 8 * (j % 2) + 2 * (j // 4) + (j // 2) % 2


def _k_place(D, j, d):
    """(byte in the tile, nibble) of element d of token j's key."""
    wc = min(4, D // 32)
    w = d // 32
    word = ((w // wc * 16 + _row(j)) * 4 + d // 8 % 4) * wc + w % wc
    return word * 4 + d % 8 // 2, d % 2


def _v_place(D, j, d):
    w = d // 16
    word = ((w // 4 * 8 + d % 8) * 4 + j // 4) * 4 + w % 4
    return 8 * D + word * 4 + j % 4, d // 8 % 2


_maps = {}


def places(D):
    """Byte and nibble of every (token, element) of a tile, for keys and values: four arrays [16, D]."""
    if D not in _maps:
        k = np.array([[_k_place(D, j, d) for d in range(D)] for j in range(16)])
        v = np.array([[_v_place(D, j, d) for d in range(D)] for j in range(16)])
        _maps[D] = (k[..., 0], k[..., 1], v[..., 0], v[..., 1])
    return _maps[D]


def _tile(cache, slot, h, D, page, group):
    off = slot % page
    n = tile_bytes(D, group)
    return cache[slot // page, h, off // 16 * n:(off // 16 + 1) * n], off % 16


def get(cache, slot, h, D, page, group):
    """((codes, scales, biases) of the key, the same of the value) of one slot and head."""
    tile, j = _tile(cache, slot, h, D, page, group)
    kb, kn, vb, vn = places(D)
    G = D // group
    coef = np.frombuffer(tile[16 * D:].tobytes(), np.float16).reshape(2, 16, G, 2)[:, _row(j)]
    return ((tile[kb[j]] >> (4 * kn[j])) & 15, coef[0, :, 0], coef[0, :, 1]), \
           ((tile[vb[j]] >> (4 * vn[j])) & 15, coef[1, :, 0], coef[1, :, 1])


def put(cache, slot, h, key, value, D, page, group):
    """Write one slot and head of `cache` in place: key and value as (codes, scales, biases)."""
    tile, j = _tile(cache, slot, h, D, page, group)
    kb, kn, vb, vn = places(D)
    G = D // group
    for (q, s, b), by, ni, part in ((key, kb[j], kn[j], 0), (value, vb[j], vn[j], 1)):
        for d in range(D):
            tile[by[d]] = (tile[by[d]] & (0xF0 if ni[d] == 0 else 0x0F)) | (int(q[d]) << (4 * ni[d]))
        for g in range(G):
            at = 16 * D + part * 64 * G + (_row(j) * G + g) * 4
            tile[at:at + 4] = np.frombuffer(np.array([s[g], b[g]], np.float16).tobytes(), np.uint8)


def values(cache, slot, D, page, group):
    """Keys and values, float64 [kv_heads, D], that one slot stands for."""
    out = []
    for part in (0, 1):
        rows = []
        for h in range(cache.shape[1]):
            q, s, b = get(cache, slot, h, D, page, group)[part]
            rows.append(q * np.repeat(s.astype(np.float64), group) + np.repeat(b.astype(np.float64), group))
        out.append(np.array(rows))
    return out


def attend(q, cache, table, lens, cu, page, group, scale, window):
    """out [T, H, D] float64 and a bound on sum_j |q||k_j| * scale and on |v| for each row's tolerance."""
    T, H, D = q.shape
    Hkv, pages = cache.shape[1], cache.shape[0]
    out = np.zeros((T, H, D))
    size = np.zeros((T, H, 2))                      # largest sum_d |q_d k_jd| * scale over j, largest |v|
    memo = {}
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        length = max(0, int(lens[b]))
        for i in range(n):
            pos = length - n + i
            js = [j for j in range(max(0, pos + 1 - window) if window else 0, min(pos + 1, length))
                  if j // page < table.shape[1] and 0 <= table[b, j // page] < pages]
            if not js:
                continue
            kv = []
            for j in js:
                slot = int(table[b, j // page]) * page + j % page
                if slot not in memo:
                    memo[slot] = values(cache, slot, D, page, group)
                kv.append(memo[slot])
            k, v = np.array([x[0] for x in kv]), np.array([x[1] for x in kv])          # [n, Hkv, D]
            for h in range(H):
                qq, kk, vv = q[cu[b] + i, h].astype(np.float64), k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
                s = kk @ qq * scale
                p = np.exp(s - s.max())
                out[cu[b] + i, h] = p @ vv / p.sum()
                size[cu[b] + i, h] = (np.abs(kk) @ np.abs(qq)).max() * scale, np.abs(vv).max()
    return out, size
