"""The 4-bit key/value cache operators on the GPU against the plain reference (kv_reference.py) and the C oracle."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build, qmm as q
    build.build()
    return q


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- plan

def run_plan(qmm, cached, fresh, free, table, tokens, page):
    cached, fresh, free = (np.array(x, np.int32) for x in (cached, fresh, free))
    t = dev(table)
    got = qmm.kv_plan(dev(cached), dev(fresh), dev(free), t, tokens, page)
    qmm.check()
    want = ref.plan(cached, fresh, free, table, tokens, page)
    for name, a, b in zip(("table", "slots", "positions", "cu", "lens", "need"), (t,) + tuple(got), want):
        assert np.array_equal(a.cpu().numpy(), b), name


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("B", [1, 3, 31, 511, 513, 1500])
def test_plan(qmm, B, page):
    rng = np.random.default_rng(B + page)
    cached, fresh = rng.integers(0, 700, B), rng.integers(0, 40, B)
    cached[rng.random(B) < 0.2] = 0
    fresh[rng.random(B) < 0.3] = 0
    cached[0] = page                                       # a full last page
    width = int((cached + fresh).max() // page) + 2
    table = rng.integers(0, 5000, (B, width)).astype(np.int32)
    free = rng.permutation(20000)[:int(sum(-(-(cached + fresh) // page)))]
    for tokens in (int(fresh.sum()), int(fresh.sum()) + 37, max(0, int(fresh.sum()) - 5)):
        run_plan(qmm, cached, fresh, free, table, tokens, page)


def test_plan_edges(qmm):
    t = np.full((2, 3), -5, np.int32)
    run_plan(qmm, [0, 0], [0, 0], [4], t, 0, 16)           # nothing to do
    run_plan(qmm, [-3, 5], [4, -1], [4, 6], t, 6, 16)      # negative lengths count as 0
    run_plan(qmm, [10, 3], [40, 60], [7], t, 100, 16)      # out of pages, and past the row's end
    run_plan(qmm, [10, 3], [40, 60], [], t, 100, 16)
    run_plan(qmm, [], [], [1], np.zeros((0, 3), np.int32), 4, 16)
    run_plan(qmm, [5], [100000], np.arange(10000) + 3, np.zeros((1, 7000), np.int32), 100000, 16)


# ---------------------------------------------------------------- append, read

def quantized(oracle_mod, x, group):
    """(codes, scales, biases) per [token, head] row from the C oracle's quantizer."""
    T, H, D = x.shape
    c, s, b = oracle_mod.quantize_affine4_f32(np.ascontiguousarray(x.reshape(T * H, D).astype(np.float32)), group)
    G = D // group
    return c.reshape(T, H, D), s.view(np.float16).reshape(T, H, G), b.view(np.float16).reshape(T, H, G)


def check_append(qmm, oracle_mod, k, v, slots, pages, page, group, dtype, strided=False):
    import torch
    T, H, D = k.shape
    rng = np.random.default_rng(7)
    before = rng.integers(0, 256, (pages, H, page // 16 * ref.tile_bytes(D, group)), dtype=np.uint8)
    cache = dev(before)
    dk, dv = dev(k.astype(np.float32)).to(dtype), dev(v.astype(np.float32)).to(dtype)
    if strided:                                            # heads of a fused projection's output
        row = torch.cat((dk, dv, dk[:, :1]), 1).contiguous()
        dk, dv = row[:, :H], row[:, H:2 * H]
    qmm.kv_append(dk, dv, dev(np.array(slots, np.int32)), cache, page, group)
    qmm.check()
    want = before.copy()
    kq = quantized(oracle_mod, dk.float().cpu().numpy(), group)
    vq = quantized(oracle_mod, dv.float().cpu().numpy(), group)
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            for h in range(H):
                ref.put(want, s, h, [x[t, h] for x in kq], [x[t, h] for x in vq], D, page, group)
    assert np.array_equal(cache.cpu().numpy(), want)       # every byte, those of no slot included
    return cache, want


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
def test_append_and_read(qmm, oracle_mod, D, group, dtype):
    import torch
    rng = np.random.default_rng(D + group)
    page, pages, H = 32, 5, 3
    for T, first in ((1, 7), (5, 30), (37, 3), (70, 64)):
        k, v = rng.standard_normal((2, T, H, D)) * rng.uniform(0.1, 3, (2, 1, 1, D))
        slots = [s % (pages * page) for s in range(first, first + T)]
        cache, want = check_append(qmm, oracle_mod, k, v, slots, pages, page, group, getattr(torch, dtype), T == 37)
        rk, rv = qmm.kv_read(dev(np.array(slots, np.int32)), cache, D, page, group)
        exact = [ref.values(want, s, D, page, group) for s in slots]
        for got, part in ((rk, 0), (rv, 1)):
            w = np.array([e[part] for e in exact]).astype(np.float32)     # s * q is exact in float32: one rounding
            assert np.array_equal(got.cpu().numpy(), w)
        bk, bv = qmm.kv_read(dev(np.array(slots, np.int32)), cache, D, page, group, dtype=torch.bfloat16)
        assert torch.equal(bk, rk.bfloat16()) and torch.equal(bv, rv.bfloat16())


@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_scattered_slots(qmm, oracle_mod, page):
    import torch
    rng = np.random.default_rng(page)
    pages, T = 6, 90
    slots = rng.permutation(pages * page)[:T].tolist() if pages * page >= T else None
    slots[5], slots[6], slots[80] = -1, pages * page, -2147483648         # skipped
    # aligned and unaligned runs inside scattered slots, reversed ones too
    slots[10:18] = [8, 9, 10, 11, 12, 13, 14, 15]
    slots[20:24] = [3, 2, 1, 0]
    slots[30:36] = [page + 6 + i for i in range(6)]
    seen = set()
    for i, s in enumerate(slots):                                          # two tokens of a call never share a slot
        if s in seen and s >= 0:
            slots[i] = -1
        seen.add(s)
    k, v = rng.standard_normal((2, T, 2, 128))
    check_append(qmm, oracle_mod, k, v, slots, pages, page, 64, torch.float32)


def test_append_edge_values(qmm, oracle_mod):
    import torch
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 1, 128)).astype(np.float32)
    x[0, 0, :64] = 0.5
    x[1, 0, :64], x[1, 0, 3] = -0.0, 0.0
    x[2, 0, 7] = np.nan
    x[3, 0, :64] = np.nan
    x[4, 0, :64] = np.float32(1e-7) * np.arange(64)
    x[5, 0, :64] = 70000.0 + np.arange(64)
    x[6, 0, 5] = np.inf
    x[7, 0, 5] = -np.inf
    j = np.arange(64) % 16
    x[8, 0, :64] = np.float32(-1.0) + j.astype(np.float32) * np.float32(0.0625)
    check_append(qmm, oracle_mod, x, x[::-1].copy(), list(range(3, 12)), 1, 16, 64, torch.float32)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("D,Hkv,T", [(64, 64, 1003), (128, 37, 1500), (256, 64, 701)])
def test_append_and_read_many_heads(qmm, D, Hkv, T, dtype):
    """Calls whose warps take several heads give the bytes and values of calls with a token each."""
    import torch
    torch.manual_seed(D)
    page, pages, group = 64, 30, 64
    k, v = torch.randn(2, T, Hkv, D, device="cuda").to(getattr(torch, dtype)).unbind(0)
    slots = torch.arange(5, T + 5, dtype=torch.int32, device="cuda")
    slots[100:140] = slots[100:140].flip(0)
    slots[200:220] = -1
    one, all_ = qmm.kv_cache(pages, Hkv, D, page, group), qmm.kv_cache(pages, Hkv, D, page, group)
    qmm.kv_append(k, v, slots, all_, page, group)
    for t in range(T):
        qmm.kv_append(k[t:t + 1], v[t:t + 1], slots[t:t + 1], one, page, group)
    assert torch.equal(one, all_) and bool(one.any())
    rk, rv = qmm.kv_read(slots, all_, D, page, group, dtype=k.dtype)
    for t in range(0, T, 7):
        for whole, part in zip((rk, rv), qmm.kv_read(slots[t:t + 1], all_, D, page, group, dtype=k.dtype)):
            assert torch.equal(whole[t].nan_to_num(7.0), part[0].nan_to_num(7.0))
    qmm.check()


def test_read_outside(qmm):
    import torch
    cache = qmm.kv_cache(2, 2, 64, 16, 64)
    k, v = qmm.kv_read(dev(np.array([-1, 3, 32, 31], np.int32)), cache, 64, 16, 64)
    for t in (k, v):
        assert torch.isnan(t[0]).all() and torch.isnan(t[2]).all() and (t[1] == 0).all() and (t[3] == 0).all()


# ---------------------------------------------------------------- attend

def make_cache(rng, pages, H, D, page, group, spread=1.0, size=1.0):
    """Random codes; scales about 0.2 and biases at -8 scales, times `size` and a factor per page spread over its decades."""
    G, tiles = D // group, page // 16
    codes = rng.integers(0, 256, (pages, H, tiles, 16 * D), dtype=np.uint8)
    f = size * spread ** rng.uniform(-1, 1, (pages, 1, 1, 1))
    s = rng.uniform(0.1, 0.3, (pages, H, tiles, 32 * G)) * f
    b = -8 * s + 0.1 * f * rng.standard_normal(s.shape)
    coef = np.ascontiguousarray(np.stack((s, b), -1).astype(np.float16)).view(np.uint8).reshape(pages, H, tiles, -1)
    return np.concatenate((codes, coef), -1).reshape(pages, H, -1)


def tolerance(size, want, lens_max, D, dtype):
    """Elementwise bound from the roundings the documentation names.

    float32: a score is a sum of D products and a few factors, each step rounded to 2^-24 of sum |q||k| * scale at
    most, the exponential's argument once more: a probability is off by twice that (numerator and denominator) plus a
    few 2^-22 of the exponential; sums over the tokens add 2^-24 a token.
    bfloat16: probabilities, keys and values may be rounded to binary16 (2^-11 each, keys enter through the score),
    the result to bfloat16 (2^-9 of itself)."""
    score, v = size[..., :1], size[..., 1:]
    if dtype == "float32":
        u = 2 * (D + 32) * 2.0 ** -24 * (score + 1) + 2.0 ** -20 + (lens_max + 64) * 2.0 ** -24
        return u * 2 * v + 1e-30
    u = 2 * 2.0 ** -10 * score + 2.0 ** -9
    return u * v + 2.0 ** -8 * np.abs(want) + 1e-30


def check_attend(qmm, rng, lens, fresh, H, Hkv, D, group, page, dtype, window=0, spread=1.0, scale=None, cu_null=False,
                 holes=False, strided=False, size=1.0):
    import torch
    B = len(lens)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 2
    cache = make_cache(rng, pages, Hkv, D, page, group, spread, size)
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((B, max(1, max(per))), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
    for b in range(B):                                     # bytes past a request's end: NaN coefficients
        if lens[b] % page:
            pg, n = table[b, per[b] - 1], ref.tile_bytes(D, group)
            tiles = cache[pg].reshape(Hkv, page // 16, n)
            G = D // group
            c = tiles[:, :, 16 * D:].copy().view(np.uint16).reshape(Hkv, page // 16, 2, 16, G, 2)
            for o in range(lens[b] % page, page):
                c[:, o // 16, :, 8 * (o % 2) + 2 * (o % 16 // 4) + (o // 2) % 2] = 0x7E00
            tiles[:, :, 16 * D:] = c.reshape(Hkv, page // 16, -1).view(np.uint8)
    if holes:
        table[rng.random(table.shape) < 0.2] = -1
        table[rng.random(table.shape) < 0.1] = pages + 3
    cu = np.concatenate(([0], np.cumsum(fresh))).astype(np.int32)
    T = int(cu[-1])
    tdt = getattr(torch, dtype)
    q = dev(rng.standard_normal((T, H, D)).astype(np.float32)).to(tdt)
    qh = q.float().cpu().numpy()
    if strided:
        q = torch.cat((q, q[:, :Hkv]), 1).contiguous()[:, :H]
    scale = D ** -0.5 if scale is None else scale
    most = max(1, max(fresh))
    ws = qmm.kv_attend_workspace(B, H, Hkv, D, most)
    out = torch.full((T, H, D), 7.0, dtype=tdt, device="cuda")
    args = (q, dev(cache), dev(table), dev(np.array(lens, np.int32)), page, group, ws)
    kw = dict(cu=None if cu_null else dev(cu), max_fresh=most, scale=scale, window=window)
    qmm.kv_attend(*args, **kw, out=out)
    qmm.check()
    assert not ws[:4096].any()
    want, sizes = ref.attend(qh, cache, table, lens, cu, page, group, scale, window)
    got = out.float().cpu().numpy().astype(np.float64)
    err, tol = np.abs(got - want), tolerance(sizes, want, max(lens), D, dtype)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"{np.max(err / tol):.2f} of the tolerance"
    again = qmm.kv_attend(*args, **kw)
    assert torch.equal(out, again)                         # the same result on every run
    return got


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (64, 64, 64), (128, 32, 32), (128, 64, 16), (128, 64, 64),
                                          (128, 128, 256), (256, 32, 16), (256, 64, 64), (256, 128, 32)])
def test_attend_one_token(qmm, D, group, page, dtype):
    rng = np.random.default_rng(D + group + page)
    check_attend(qmm, rng, [1, 0, 2, 15, 16, 17, 33, 130], [1] * 8, 4, 2, D, group, page, dtype)
    check_attend(qmm, rng, [300, 31], [1, 1], 3, 3, D, group, page, dtype, cu_null=True, strided=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("ratio", [1, 2, 5, 7, 8, 9, 12, 16, 24, 33])
def test_attend_head_groups(qmm, ratio, dtype):
    rng = np.random.default_rng(ratio)
    check_attend(qmm, rng, [70, 5, 129], [1, 1, 1], 2 * ratio, 2, 64, 64, 16, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("window", [0, 1, 20, 64])
def test_attend_several_tokens(qmm, window, dtype):
    rng = np.random.default_rng(window)
    for D, group in ((64, 32), (128, 64), (256, 64)):
        check_attend(qmm, rng, [40, 0, 3, 90, 7], [5, 2, 3, 1, 0], 6, 2, D, group, 16, dtype, window=window)
        check_attend(qmm, rng, [3, 50], [5, 4], 4, 1, D, group, 32, dtype, window=window)     # queries before the start


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("D,group,page", [(64, 64, 16), (128, 64, 64), (128, 32, 16), (256, 64, 32), (256, 128, 16)])
def test_attend_prompts(qmm, D, group, page, dtype):
    rng = np.random.default_rng(D + page)
    check_attend(qmm, rng, [130, 61, 200, 0, 1], [130, 33, 65, 0, 1], 4, 2, D, group, page, dtype)
    check_attend(qmm, rng, [150, 140], [140, 40], 3, 1, D, group, page, dtype, window=37, strided=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attend_long_context(qmm, dtype):
    """Splits over many blocks, with one long and many short requests."""
    rng = np.random.default_rng(17)
    check_attend(qmm, rng, [5000] + [9] * 20, [1] * 21, 2, 1, 64, 64, 64, dtype)
    check_attend(qmm, rng, [2100, 3], [3, 2], 8, 1, 128, 64, 16, dtype, window=700)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attend_missing_pages(qmm, dtype):
    rng = np.random.default_rng(23)
    check_attend(qmm, rng, [200, 90, 16], [1, 1, 1], 4, 2, 128, 64, 16, dtype, holes=True)
    check_attend(qmm, rng, [180, 150], [40, 70], 4, 2, 64, 64, 16, dtype, holes=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attend_scales_over_many_decades(qmm, dtype):
    """Pages whose coefficients differ by up to a factor of 1e6 from one another: the largest must not cost the rest."""
    rng = np.random.default_rng(29)
    check_attend(qmm, rng, [400, 65], [1, 1], 4, 2, 128, 64, 16, dtype, spread=1e3, scale=0.01)
    check_attend(qmm, rng, [120], [90], 4, 2, 128, 64, 16, dtype, spread=1e3, scale=0.01)


def many_rows(D):
    """Rows of q of all requests and kv heads beyond which a bfloat16 call's prompts fill the GPU with tiles of them."""
    return {64: 8700, 128: 7400, 256: 4000}[D]


@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (64, 64, 64), (128, 32, 32), (128, 64, 16), (128, 64, 256),
                                          (128, 128, 64), (256, 32, 128), (256, 64, 64), (256, 128, 16)])
def test_attend_many_rows(qmm, D, group, page):
    rng = np.random.default_rng(D + group + page)
    assert 5 * 130 * 16 > many_rows(D) and 280 * 33 > many_rows(D)
    check_attend(qmm, rng, [130, 61, 200, 0, 1], [130, 33, 65, 0, 1], 16, 2, D, group, page, "bfloat16")
    check_attend(qmm, rng, [150, 140], [140, 40], 33, 1, D, group, page, "bfloat16", window=37, strided=True)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
def test_attend_many_rows_of_few_tokens(qmm, D, group):
    """One partly filled tile a request and head, some requests empty, some with queries before their start."""
    rng = np.random.default_rng(D)
    fresh = [8] + rng.integers(0, 9, 29).tolist()
    lens = rng.integers(0, 150, 30).tolist()
    lens[3], lens[7] = 0, 3
    assert 30 * 5 * 64 > many_rows(D)
    check_attend(qmm, rng, lens, fresh, 40, 5, D, group, 32, "bfloat16")
    check_attend(qmm, rng, lens, fresh, 40, 5, D, group, 16, "bfloat16", window=5, holes=True)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 128)])
def test_attend_many_rows_small_large_and_missing(qmm, D, group):
    rng = np.random.default_rng(D + 1)
    case = ([260, 90], [130, 60], 64, 2, D, group, 16, "bfloat16")
    check_attend(qmm, rng, *case, holes=True)
    check_attend(qmm, rng, *case, spread=1e3, scale=0.01)               # scales up to 300
    check_attend(qmm, rng, *case, spread=1.0, scale=2.0 * D ** -0.5)    # peaked: the maxima keep growing
    check_attend(qmm, rng, *case, size=2.0 ** -8, scale=256 * D ** -0.5)   # keys and values of 0.004


@pytest.mark.parametrize("H,Hkv", [(4, 2), (64, 2)])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attend_non_finite_values(qmm, D, group, H, Hkv, dtype):
    """A value whose coefficients are not finite reaches the queries that see it, its head and its group, nothing else;
    an infinite key is as good as any where it is not seen."""
    import torch
    rng = np.random.default_rng(D + H)
    page, n, length, G = 16, 140, 150, D // group
    cache = make_cache(rng, 12, Hkv, D, page, group)
    table = rng.permutation(12).astype(np.int32)[None, :10]
    clean = cache.copy()

    def coef(token, head, part, g, k):
        tile = cache[table[0, token // page], head].reshape(page // 16, -1)[token % page // 16]
        at = 16 * D + part * 64 * G + ((8 * (token % 2) + 2 * (token % 16 // 4) + (token // 2) % 2) * G + g) * 4 + 2 * k
        return tile[at:at + 2].view(np.uint16)

    spots = [(77, 1, G - 1), (139, 0, 0)]                   # token, head, group
    first, ratio = length - n, H // Hkv
    q = dev(rng.standard_normal((n, H, D)).astype(np.float32)).to(getattr(torch, dtype))
    cu = np.array([0, n], np.int32)
    want, sizes = ref.attend(q.float().cpu().numpy(), clean, table, [length], cu, page, group, D ** -0.5, 0)
    tol = np.broadcast_to(tolerance(sizes, want, length, D, dtype), want.shape)
    hit = np.zeros(want.shape, bool)
    for token, head, g in spots:
        hit[token - first:, head * ratio:(head + 1) * ratio, g * group:(g + 1) * group] = True
    rest = ~hit
    rest[-1, :ratio] = False                                # what an infinite key does to the query that sees it is not
    hit[-1, :ratio] = False                                 # looked at
    ws = qmm.kv_attend_workspace(1, H, Hkv, D, n)
    for k, bits in ((0, 0x7E01), (1, 0x7C00), (0, 0x7C00)):     # a NaN scale, an infinite bias, an infinite scale
        cache[:] = clean
        for token, head, g in spots:
            coef(token, head, 1, g, k)[:] = bits
        coef(149, 0, 0, 0, 1)[:] = 0x7C00                   # the last key: seen by the last query alone
        got = qmm.kv_attend(q, dev(cache), dev(table), dev(np.array([length], np.int32)), page, group, ws, cu=dev(cu),
                            max_fresh=n).float().cpu().numpy()
        qmm.check()
        assert not np.isfinite(got[hit]).any()
        assert (np.abs(got - want)[rest] <= tol[rest]).all()


def test_large_cache(qmm):
    """Pages beyond 4 GiB of a cache hold and give what pages at its start do."""
    import torch
    page, Hkv, D, group, n = 256, 8, 128, 64, 1300
    pages = (1 << 32) // (Hkv * (page // 16) * ref.tile_bytes(D, group)) + 40
    cache = qmm.kv_cache(pages, Hkv, D, page, group)
    torch.manual_seed(5)
    k, v = torch.randn(2, n, Hkv, D, device="cuda").unbind(0)
    cu, lens, ws = dev(np.array([0, n], np.int32)), dev(np.array([n], np.int32)), qmm.kv_attend_workspace(1, 32, Hkv, D, n)
    got = []
    for first in (0, pages - 6):
        table = torch.arange(first, first + 6, dtype=torch.int32, device="cuda")[None].contiguous()
        slots = first * page + torch.arange(n, dtype=torch.int32, device="cuda")
        qmm.kv_append(k, v, slots, cache, page, group)
        outs = list(qmm.kv_read(slots, cache, D, page, group))
        for dtype in (torch.float32, torch.bfloat16):
            torch.manual_seed(6)
            q = torch.randn(n, 32, D, device="cuda").to(dtype)
            outs.append(qmm.kv_attend(q, cache, table, lens, page, group, ws, cu=cu, max_fresh=n))
            outs.append(qmm.kv_attend(q[:1], cache, table, lens, page, group, ws))
        qmm.check()
        got.append(outs)
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert all(bool((x != 0).any()) for x in got[1])


def test_attend_more_requests_than_threads(qmm):
    rng = np.random.default_rng(31)
    lens = rng.integers(0, 40, 1300).tolist()
    check_attend(qmm, rng, lens, [1] * 1300, 1, 1, 64, 64, 16, "float32")


def test_attend_nan_stays_in_its_request(qmm):
    """A NaN coefficient inside one request reaches that request's output and no other's."""
    import torch
    rng = np.random.default_rng(37)
    cache = make_cache(rng, 4, 1, 64, 16, 64)
    cache[2].reshape(-1)[16 * 64:16 * 64 + 64].view(np.uint16)[0] = 0x7E00     # K scale of row 0, page 2
    table = np.array([[0, 1], [2, 3]], np.int32)
    q = dev(rng.standard_normal((2, 1, 64)).astype(np.float32))
    ws = qmm.kv_attend_workspace(2, 1, 1, 64)
    out = qmm.kv_attend(q, dev(cache), dev(table), dev(np.array([30, 30], np.int32)), 16, 64, ws)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


def test_steps_together_on_a_side_stream(qmm, oracle_mod):
    """plan, append and attend chained on a stream of their own, in a captured graph replayed with new lengths."""
    import torch
    rng = np.random.default_rng(41)
    B, H, Hkv, D, page, group, pages = 3, 4, 2, 64, 16, 64, 24
    cache = qmm.kv_cache(pages, Hkv, D, page, group)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    cached = torch.zeros(B, dtype=torch.int32, device="cuda")
    fresh = torch.ones(B, dtype=torch.int32, device="cuda")
    order = rng.permutation(pages).astype(np.int32)
    free = dev(order)
    k, v, q = (torch.zeros(B, n, D, device="cuda") for n in (Hkv, Hkv, H))
    ws = qmm.kv_attend_workspace(B, H, Hkv, D)

    def step():
        slots, positions, cu, lens, need = qmm.kv_plan(cached, fresh, free, table, B, page)
        qmm.kv_append(k, v, slots, cache, page, group)
        return qmm.kv_attend(q, cache, table, lens, page, group, ws, cu=cu), need

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    cache.zero_(), table.fill_(-1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, need = step()
    taken, hist = 0, []
    for n in range(40):
        kk, vv, qq = (rng.standard_normal(t.shape).astype(np.float32) for t in (k, v, q))
        k.copy_(dev(kk)), v.copy_(dev(vv)), q.copy_(dev(qq))
        cached.fill_(n)
        free.copy_(dev(np.roll(order, -taken)))
        graph.replay()
        torch.cuda.synchronize()
        taken += int(need)
        hist.append((kk, vv))
        if n in (0, 15, 16, 39):
            host, tab = cache.cpu().numpy(), table.cpu().numpy()
            want, size = ref.attend(qq, host, tab, [n + 1] * B, np.arange(B + 1), page, group, D ** -0.5, 0)
            err = np.abs(out.cpu().numpy() - want)
            assert (err <= tolerance(size, want, n + 1, D, "float32")).all()
            for t in range(n + 1):                         # and the cache holds what was appended
                kq = quantized(oracle_mod, hist[t][0], group)
                for b in range(B):
                    got = ref.get(host, int(tab[b, t // page]) * page + t % page, 1, D, page, group)[0]
                    assert np.array_equal(got[0], kq[0][b, 1])
    assert taken == 3 * 3
