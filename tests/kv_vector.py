"""The attention of kv_reference.py over whole arrays at a time (float64 torch, on the GPU where there is one), for cases of
thousands of queries.  The layout is kv_reference.py's, element by element."""
import numpy as np
import torch

import kv_reference as ref


def decode(cache, D, page, group):
    """Keys and values, float64 [pages, kv_heads, page, D], that a cache (numpy) stands for."""
    P, H = cache.shape[:2]
    G, tiles = D // group, cache.reshape(P, H, page // 16, -1)
    kb, kn, vb, vn = ref.places(D)
    rows = [ref._row(j) for j in range(16)]
    coef = np.ascontiguousarray(tiles[..., 16 * D:]).view(np.float16).reshape(P, H, page // 16, 2, 16, G, 2)[..., rows, :, :]
    out = []
    for part, by, ni in ((0, kb, kn), (1, vb, vn)):
        q = (tiles[..., by] >> (4 * ni).astype(np.uint8)) & 15
        c = np.repeat(coef[:, :, :, part].astype(np.float64), group, -2)
        with np.errstate(invalid="ignore"):
            out.append((q * c[..., 0] + c[..., 1]).reshape(P, H, page, D))
    return out


def attend(q, k, v, table, lens, cu, page, scale, window):
    """out and sizes as in kv_reference.attend: q [T, H, D] numpy, k and v [pages, kv_heads, page, D] float64 numpy."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    T, H, D = q.shape
    P, Hkv = k.shape[:2]
    q, k, v = (torch.from_numpy(np.asarray(x, np.float64)).to(dev) for x in (q, k, v))
    out = torch.zeros((T, H, D), dtype=torch.float64, device=dev)
    size = torch.zeros((T, H, 2), dtype=torch.float64, device=dev)
    for b in range(len(lens)):
        n, length = int(cu[b + 1] - cu[b]), max(0, int(lens[b]))
        js = np.arange(min(length, table.shape[1] * page))
        pg = table[b, js // page]
        there = (pg >= 0) & (pg < P)
        js, pg = js[there], pg[there]
        if n == 0 or len(js) == 0:
            continue
        pos = length - n + np.arange(n)[:, None]
        seen = (js <= pos) & ((js > pos - window) if window else True)
        at = torch.from_numpy(pg.astype(np.int64)).to(dev), torch.from_numpy(js % page).to(dev)
        kk, vv = (x[at[0], :, at[1]] for x in (k, v))                          # [J, Hkv, D]
        seen = torch.from_numpy(seen).to(dev)
        x = q[cu[b]:cu[b + 1]].view(n, Hkv, H // Hkv, D)
        s = torch.einsum("nhrd,jhd->hrnj", x, kk) * scale
        s = s.masked_fill(~seen, float("-inf"))
        p = torch.softmax(s, -1).nan_to_num(0.0)
        out[cu[b]:cu[b + 1]] = torch.einsum("hrnj,jhd->nhrd", p, vv).reshape(n, H, D)
        big = torch.einsum("nhrd,jhd->hrnj", x.abs(), kk.abs()) * scale
        size[cu[b]:cu[b + 1], :, 0] = big.masked_fill(~seen, 0.0).amax(-1).permute(2, 0, 1).reshape(n, H)
        most = vv.abs().amax(-1).t()[:, None].expand(Hkv, n, len(js)).masked_fill(~seen, 0.0).amax(-1)
        size[cu[b]:cu[b + 1], :, 1] = most.t().repeat_interleave(H // Hkv, 1)
    return out.cpu().numpy(), size.cpu().numpy()
