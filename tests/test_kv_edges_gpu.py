"""The 4-bit key/value cache operators at the ends of what they accept."""
import numpy as np
import pytest

import kv_vector as vec
from test_kv_gpu import dev, make_cache, run_plan, tolerance
from test_kv_items_gpu import check_items, takes_tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build, qmm as q
    build.build()
    return q


class Case:
    """One request of `length` tokens, the last n of which ask; H = 64 over 2 kv heads are rows enough for the prompt kernel."""

    def __init__(self, seed, D, group, H, dtype, n=140, length=150, page=16, Hkv=2):
        import torch
        rng = np.random.default_rng(seed)
        self.D, self.group, self.H, self.Hkv, self.n, self.length, self.page, self.dtype = D, group, H, Hkv, n, length, page, dtype
        blocks = -(-length // page)
        self.cache = make_cache(rng, blocks + 2, Hkv, D, page, group)
        self.table = rng.permutation(blocks + 2).astype(np.int32)[None, :blocks]
        self.q = dev(rng.standard_normal((n, H, D)).astype(np.float32)).to(getattr(torch, dtype))

    def coef(self, token, head, value, g):
        """[scale, bias] of a token's key or value as binary16 bits, to be written."""
        tile = self.cache[self.table[0, token // self.page], head].reshape(self.page // 16, -1)[token % self.page // 16]
        G = self.D // self.group
        at = 16 * self.D + value * 64 * G + ((8 * (token % 2) + 2 * (token % 16 // 4) + (token // 2) % 2) * G + g) * 4
        return tile[at:at + 4].view(np.uint16)

    def want(self, scale=None, window=0, cache=None):
        """(out, tolerance) in 64 bits."""
        scale = self.D ** -0.5 if scale is None else scale
        k, v = vec.decode(self.cache if cache is None else cache, self.D, self.page, self.group)
        want, sizes = vec.attend(self.q.float().cpu().numpy(), k, v, self.table, [self.length], [0, self.n], self.page, scale,
                                 window)
        return want, np.broadcast_to(tolerance(sizes, want, self.length, self.D, self.dtype), want.shape)

    def run(self, qmm, scale=None, window=0, out=None):
        ws = qmm.kv_attend_workspace(1, self.H, self.Hkv, self.D, self.n)
        out = qmm.kv_attend(self.q, dev(self.cache), dev(self.table), dev(np.array([self.length], np.int32)), self.page,
                            self.group, ws, cu=dev(np.array([0, self.n], np.int32)), max_fresh=self.n, scale=scale, window=window,
                            out=out)
        qmm.check()
        assert not ws[:4096].any()
        return out.float().cpu().numpy().astype(np.float64)


ROUTES = [(4, "float32"), (4, "bfloat16"), (64, "float32"), (64, "bfloat16")]
NAN, INF, MINUS_INF = 0x7E01, 0x7C00, 0xFC00


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 64), (128, 128), (256, 32), (256, 128)])
def test_finite_values_beyond_binary16(qmm, D, group, H, dtype, window):
    """Finite coefficients whose values pass 65504: finite outputs everywhere, and queries that do not see them as exact as ever."""
    c = Case(D + H, D, group, H, dtype)
    G = D // group
    for token, head, g, s, b in ((149, 0, 0, 5332, 0), (149, 1, G - 1, 65504, 65504), (131, 0, G - 1, -5332, 0),
                                 (64, 1, 0, 8000, -60000), (9, 0, 0, 65504, -65504)):
        c.coef(token, head, 1, g)[:] = np.array([s, b], np.float16).view(np.uint16)
    want, tol = c.want(window=window)
    got = c.run(qmm, window=window)
    assert np.isfinite(got).all()
    # bounds by element: |v| of the groups that hold large values would hide the others
    k, v = vec.decode(c.cache, D, c.page, group)
    for g in range(G):
        part = slice(g * group, (g + 1) * group)
        _, sizes = vec.attend(c.q.float().cpu().numpy(), k, np.where(np.arange(D) // group == g, v, 0.0), c.table, [c.length],
                              [0, c.n], c.page, D ** -0.5, window)
        bound = tolerance(sizes, want[..., part], c.length, D, dtype)
        assert (np.abs(got - want)[..., part] <= bound).all(), g


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 64)])
def test_finite_values_beyond_binary16_in_some_of_many_items(qmm, D, group):
    """Items with such values and without, one after the other on every SM."""
    rng = np.random.default_rng(D)
    B, H, Hkv, page = 80, 32, 8, 32
    fresh = [20 if b % 2 else 64 for b in range(B)]
    lens = rng.integers(64, 300, B).tolist()

    def change(cache, table):
        tiles = cache.reshape(len(cache), Hkv, page // 16, -1)
        coef = tiles[..., 16 * D + 64 * (D // group):].reshape(len(cache), Hkv, -1)
        for b in range(0, B, 3):
            row = table[b, int(rng.integers(0, lens[b] // page))], int(rng.integers(0, Hkv))
            coef[row][4:8].view(np.float16)[:] = 65504, -30000
        tiles[..., 16 * D + 64 * (D // group):] = coef.reshape(len(cache), Hkv, page // 16, -1)

    assert takes_tiles(B, H, Hkv, D, 64)
    check_items(qmm, rng, lens, fresh, H, Hkv, D, group, page, "bfloat16", runs=5, change=change)


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 128)])
def test_finite_keys_beyond_binary16(qmm, D, group, H, dtype):
    c = Case(D + H, D, group, H, dtype)
    for token, head, g, s, b in ((149, 0, 0, 5332, 0), (100, 1, 0, 65504, 65504), (64, 1, D // group - 1, 8000, -60000)):
        c.coef(token, head, 0, g)[:] = np.array([s, b], np.float16).view(np.uint16)
    want, tol = c.want(scale=1e-7)
    assert (np.abs(c.run(qmm, scale=1e-7) - want) <= tol).all()


@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 64)])
@pytest.mark.parametrize("sink", [9.0, 12.3, 14.2])
def test_many_small_probabilities_beside_a_large_one(qmm, D, group, sink):
    """One key takes nearly all the weight and its value is zero: the output is what 65535 tokens of e^-sink each add up to.
    Their keys are zero and their values positive, so that the roundings of P (2^-11) and of the values (2^-11) bound the error
    of each element before it is rounded to the output's type; float32 sums and factors stay below 2^-14."""
    import torch
    n, length, page, H, Hkv, G = 128, 65536, 256, 72, 2, D // group
    assert Hkv * n * H // Hkv > 8000                       # the prompt kernel
    rng = np.random.default_rng(D)
    tiles = length // 16
    codes = rng.integers(0, 256, (tiles, Hkv, 16 * D), dtype=np.uint8)
    coef = np.zeros((tiles, Hkv, 2, 16, G, 2), np.float16)
    coef[:, :, 1, ..., 0] = rng.uniform(0.01, 0.06, (tiles, Hkv, 16, G))
    coef[:, :, 1, ..., 1] = rng.uniform(0.3, 0.6, (tiles, Hkv, 16, G))
    coef[0, :, 0, 0, :, 1] = 1.0                           # token 0: a key of ones, a value of zeros
    coef[0, :, 1, 0] = 0.0
    cache = np.concatenate((codes, coef.view(np.uint8).reshape(tiles, Hkv, -1)), -1)
    cache = np.ascontiguousarray(cache.reshape(length // page, page // 16, Hkv, -1).transpose(0, 2, 1, 3)).reshape(
        length // page, Hkv, -1)
    table = rng.permutation(length // page).astype(np.int32)
    held = np.empty_like(cache)
    held[table] = cache
    q = dev((rng.uniform(0.9, 1.1, (n, H, D)) * sink * D ** -0.5).astype(np.float32)).bfloat16()
    out = qmm.kv_attend(q, dev(held), dev(table[None]), dev(np.array([length], np.int32)), page, group,
                        qmm.kv_attend_workspace(1, H, Hkv, D, n), cu=dev(np.array([0, n], np.int32)), max_fresh=n)
    qmm.check()
    _, v = vec.decode(cache, D, page, group)
    v = torch.from_numpy(v).cuda().transpose(1, 2).reshape(length, Hkv, D)
    upto = torch.cumsum(v, 0)[length - n:]                 # [n, Hkv, D]: sums of what each query sees
    score = torch.exp(q.double().sum(-1) * D ** -0.5)      # the first key's weight beside ones
    count = torch.arange(length - n, length, device="cuda")[:, None] + score
    want = upto.repeat_interleave(H // Hkv, 1) / count[..., None]
    off = 2 * 2.0 ** -11 + 2.0 ** -14
    low, high = ((want * (1 + x)).to(out.dtype) for x in (-off, off))
    assert bool(((low <= out) & (out <= high)).all()), f"{float(((out.double() - want).abs() / want).max()):.5f}"


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 64), (128, 32), (256, 64), (256, 128)])
def test_keys_that_are_not_finite(qmm, D, group, H, dtype):
    """Every query that sees such a key gets nothing finite, whichever the signs of its elements; no other is touched."""
    c = Case(D + H, D, group, H, dtype)
    c.q[::2] = c.q[::2].abs()                              # the sum over a group has one sign: a score of -inf alone
    c.q[1::4] = -c.q[1::4].abs()
    want, tol = c.want()
    clean = c.cache.copy()
    ratio, first = H // 2, c.length - c.n
    for token, head, g in ((77, 1, D // group - 1), (149, 0, 0)):
        hit = np.zeros(want.shape[:2], bool)
        hit[token - first:, head * ratio:(head + 1) * ratio] = True
        for k, bits in ((1, MINUS_INF), (1, INF), (0, INF), (0, MINUS_INF), (0, NAN), (1, NAN)):
            c.cache[:] = clean
            c.coef(token, head, 0, g)[k] = bits
            got = c.run(qmm)
            assert not np.isfinite(got[hit]).any(), (token, k, hex(bits))
            assert (np.abs(got - want)[~hit] <= tol[~hit]).all(), (token, k, hex(bits))


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_values_that_are_not_finite_at_no_weight(qmm, D, group, H, dtype):
    """Such a value reaches its group of every query that sees it, however small the probability."""
    c = Case(D + H, D, group, H, dtype)
    c.q[:] = c.q.abs()
    ratio, first, G = H // 2, c.length - c.n, D // group
    spots = [(77, 1, G - 1), (139, 0, 0), (5, 0, G - 1)]
    for token, head, g in spots:
        for i in range(G):
            c.coef(token, head, 0, i)[:] = np.array([0.0, -1000.0], np.float16).view(np.uint16)    # exp() of it is 0
    want, tol = c.want()
    clean = c.cache.copy()
    for k, bits in ((1, INF), (0, INF), (0, NAN)):
        c.cache[:] = clean
        hit = np.zeros(want.shape, bool)
        for token, head, g in spots:
            c.coef(token, head, 1, g)[k] = bits
            hit[max(0, token - first):, head * ratio:(head + 1) * ratio, g * group:(g + 1) * group] = True
        got = c.run(qmm)
        assert not np.isfinite(got[hit]).any(), (k, hex(bits))
        assert (np.abs(got - want)[~hit] <= tol[~hit]).all(), (k, hex(bits))


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_underflow(qmm, D, H, dtype):
    """The least queries and scales: all scores are 0 in float32, so the outputs are means of what is seen."""
    c = Case(D, D, 64, H, dtype)
    c.q.mul_(2e-38)
    want, tol = c.want(scale=1e-30)
    got = c.run(qmm, scale=1e-30)
    assert (np.abs(got - want) <= tol).all()


def test_missing_pages_past_2_30_tokens(qmm):
    """Positions beyond 2^30: a page that is not there is left out there, too."""
    import torch
    page, length, window, n, D, group, H, Hkv = 256, (1 << 30) + 300, 600, 140, 64, 64, 64, 2
    rng = np.random.default_rng(3)
    cache = make_cache(rng, 4, Hkv, D, page, group)
    blocks = -(-length // page)
    table = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.tensor([2, 1], dtype=torch.int32)
    table[0, -4] = 3                                       # positions 2^30 - 512 .. 2^30 - 257; the page after it is missing
    for dtype in ("float32", "bfloat16"):
        q = dev(rng.standard_normal((n, H, D)).astype(np.float32)).to(getattr(torch, dtype))
        out = qmm.kv_attend(q, dev(cache), table, dev(np.array([length], np.int32)), page, group,
                            qmm.kv_attend_workspace(1, H, Hkv, D, n), cu=dev(np.array([0, n], np.int32)), max_fresh=n,
                            window=window)
        qmm.check()
        short = np.array([[3, -1, 2, 1]], np.int32)        # the same tokens without what lies before them
        want, sizes = vec.attend(q.float().cpu().numpy(), *vec.decode(cache, D, page, group), short,
                                 [length - (blocks - 4) * page], [0, n], page, D ** -0.5, window)
        assert (np.abs(out.float().cpu().numpy() - want) <= tolerance(sizes, want, 1024, D, dtype)).all(), dtype


@pytest.mark.parametrize("B", [6112, 6113, 6144, 6145, 8192])
def test_plan_of_wide_batches(qmm, B):
    rng = np.random.default_rng(B)
    cached, fresh = rng.integers(0, 60, B), rng.integers(0, 3, B)
    table = rng.integers(0, 5000, (B, 5)).astype(np.int32)
    run_plan(qmm, cached, fresh, rng.permutation(9000), table, int(fresh.sum()) + 3, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_empty_cache(qmm, D):
    """A cache without pages takes every call: nothing is kept, nothing is seen."""
    import torch
    H, Hkv, n, page = 64, 2, 140, 16
    cache = qmm.kv_cache(0, Hkv, D, page)
    k, slots = torch.randn(n, Hkv, D, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    qmm.kv_append(k, k, slots, cache, page)
    for x in qmm.kv_read(slots, cache, D, page):
        assert bool(x.isnan().all())
    lens, cu = dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32))
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn(n, H, D, device="cuda").to(dtype)
        for table in (torch.zeros(1, 9, dtype=torch.int32, device="cuda"), torch.zeros(1, 0, dtype=torch.int32, device="cuda")):
            out = qmm.kv_attend(q, cache, table, lens, page, 64, qmm.kv_attend_workspace(1, H, Hkv, D, n), cu=cu, max_fresh=n,
                                out=torch.full_like(q, 7.0))
            assert not bool(out.any())
    qmm.check()


def heads_first(x):
    """The same [tokens, heads, head_dim] tensor, laid out as [heads, tokens, head_dim]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_heads_first(qmm, D, H, dtype):
    c = Case(D + 1, D, 64, H, dtype)
    plain = c.run(qmm)
    c.q = heads_first(c.q)
    assert c.q.stride(0) == D and np.array_equal(c.run(qmm), plain)
    want, tol = c.want()
    assert (np.abs(plain - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 50, 700])
def test_append_heads_first(qmm, T, dtype):
    import torch
    torch.manual_seed(T)
    k, v = torch.randn(2, T, 24, 128, device="cuda").to(getattr(torch, dtype)).unbind(0)
    slots = torch.randperm(T + 9, device="cuda")[:T].int()
    caches = [qmm.kv_cache(T // 32 + 2, 24, 128, 32) for _ in range(2)]
    qmm.kv_append(k, v, slots, caches[0], 32)
    qmm.kv_append(heads_first(k), heads_first(v), slots, caches[1], 32)
    assert torch.equal(*caches) and bool(caches[0].any())
    shared = v[:, :1].expand(-1, 24, -1)                   # one value head for all key heads: a head stride of 0
    qmm.kv_append(k, shared, slots, caches[0], 32)
    qmm.kv_append(k, shared.contiguous(), slots, caches[1], 32)
    assert torch.equal(*caches)


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_output_over_the_queries(qmm, D, H, dtype):
    """out may be q, where an item is done twice for its large values, too."""
    c = Case(D + 2, D, 64, H, dtype)
    for large in (False, True):
        if large:
            c.coef(100, 1, 1, 0)[:] = np.array([65504, -30000], np.float16).view(np.uint16)
        want = c.run(qmm)
        held = c.q.clone()
        assert np.array_equal(c.run(qmm, out=c.q), want)
        c.q = held


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_that_are_not_finite(qmm, D, H, dtype):
    """They reach their own output and no other."""
    c = Case(D + 3, D, 64, H, dtype)
    want, tol = c.want()
    hit = np.zeros(want.shape[:2], bool)
    for token, head, value in ((0, 0, np.nan), (70, H - 1, np.inf), (139, H // 2, -np.inf)):
        c.q[token, head, 3] = value
        hit[token, head] = True
    got = c.run(qmm)
    assert not np.isfinite(got[hit]).any()
    assert (np.abs(got - want)[~hit] <= tol[~hit]).all()


@pytest.mark.parametrize("H,dtype", ROUTES)
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (128, 128), (256, 32)])
def test_scales_of_either_sign(qmm, D, group, H, dtype):
    """Small negative scales beside large positive ones, and the other way round."""
    for sign in (1, -1):
        c = Case(D + group, D, group, H, dtype)
        rng = np.random.default_rng(D)
        coef = c.cache.reshape(len(c.cache), 2, -1)[:, :, 16 * D:].copy().view(np.float16)      # one tile a page
        s = coef[..., ::2]
        s *= np.where(rng.random(s.shape) < 0.5, -1.0, 1.0).astype(np.float16)
        c.cache.reshape(len(c.cache), 2, -1)[:, :, 16 * D:] = coef.view(np.uint8)
        for token in range(0, c.length, 7):
            c.coef(token, token % 2, 1, token % (D // group))[:] = np.array([sign * 900.0, -100.0], np.float16).view(np.uint16)
        want, tol = c.want()
        assert (np.abs(c.run(qmm) - want) <= tol).all(), sign
