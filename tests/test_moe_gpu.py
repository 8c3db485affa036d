"""The routing of tokens to experts, the experts' products and the way back, against float64."""
import numpy as np
import pytest

import mx4_reference as ref
from test_mx4_gpu import T, check_product, matrix, on_gpu, qmm, spread  # noqa: F401

pytestmark = pytest.mark.gpu


def plan_of(logits, k, normalize):
    """experts, weights, places, starts, counts of float64 logits."""
    n, E = logits.shape
    experts, weights = np.full((n, k), -1), np.zeros((n, k))
    lists = [[] for _ in range(E)]
    for t, row in enumerate(logits):
        rank = sorted(range(E), key=lambda e: (not np.isnan(row[e]), -row[e] if not np.isnan(row[e]) else 0, e))
        take = [e for e in rank[:k] if row[e] != -np.inf]
        if not take:
            continue
        with np.errstate(invalid="ignore"):
            p = np.exp(row[take] - row[take[0]])
            whole = p.sum() if normalize else np.exp(row[row != -np.inf] - row[take[0]]).sum()
            weights[t, :len(take)] = p / whole
        experts[t, :len(take)] = take
        for j, e in enumerate(take):
            lists[e].append((t, j))
    counts = np.array([len(l) for l in lists])
    starts = np.concatenate(([0], np.cumsum((counts + 127) // 128 * 128)[:-1]))
    places = np.full((n, k), -1)
    for e, l in enumerate(lists):
        for i, (t, j) in enumerate(l):
            places[t, j] = starts[e] + i
    return experts, weights, places, starts, counts


def check_plan(got, want, E):
    for g, w in zip((got[0], got[2], got[3], got[4]), (want[0], want[2], want[3], want[4])):
        assert np.array_equal(g.cpu().numpy(), w)
    # an exponential and a sum of E of them: 2 ulp and E / 2 roundings, two more for the quotient
    w, g = want[1], got[1].cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(w))
    # (the difference of two logits is rounded once, and its error is the exponential's relative one)
    assert np.allclose(g, w, rtol=(8 + E / 2) * 2.0 ** -23, atol=2.0 ** -126, equal_nan=True)


@pytest.mark.parametrize("n,E,k", [(0, 5, 2), (1, 1, 1), (1, 64, 6), (7, 3, 3), (8, 64, 8), (33, 33, 4), (64, 100, 32), (65, 8, 2),
                                   (200, 128, 8), (513, 256, 1), (700, 1024, 5), (1000, 17, 4), (3001, 60, 6), (5000, 2, 2)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("normalize", [True, False])
def test_plan(T, qmm, n, E, k, dtype, normalize):
    rng = np.random.default_rng(n * 1000 + E)
    l = T.from_numpy(rng.standard_normal((n, E)) * 2 + rng.standard_normal(E)).to(getattr(T, dtype)).cuda()
    got = qmm.moe_plan(l, k, normalize=normalize)
    qmm.check()
    check_plan(got, plan_of(l.double().cpu().numpy(), k, normalize), E)
    used = got[2].flatten()
    assert n == 0 or int(used.max()) < qmm.moe_rows(n, E, k)


@pytest.mark.parametrize("n", [50, 700])
@pytest.mark.parametrize("normalize", [True, False])
def test_plan_of_ties_masks_and_what_is_not_finite(T, qmm, n, normalize):
    E, k = 40, 6
    rng = np.random.default_rng(n)
    l = rng.integers(-2, 3, (n, E)).astype(np.float32)           # ties everywhere
    l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, -0.0, 0.0)
    l[1] = -np.inf                                               # a token with no expert
    l[2, :] = -np.inf
    l[2, [5, 30]] = [1.0, 2.0]                                   # with two
    l[3] = np.finfo(np.float32).min                              # the lowest value is no mask
    l[4, 7] = np.inf
    l[5, [3, 20]] = np.nan
    l[6] = np.nan
    l[7, ::2] = -np.inf
    l[8, 1:] = np.finfo(np.float32).min
    got = qmm.moe_plan(T.from_numpy(l).cuda(), k, normalize=normalize)
    qmm.check()
    want = plan_of(l.astype(np.float64), k, normalize)
    want[1][4] = np.nan                                          # an infinity less itself, as softmax has it
    if normalize:
        want[1][3] = 1 / k
    else:
        want[1][3] = 1 / E
    check_plan(got, want, E)


def test_plan_all_to_one_expert_and_strides(T, qmm):
    n, E = 4000, 12
    full = T.zeros(n, 20, device="cuda")
    full[:, 3 + 4] = 5.0
    l = full[:, 3:15]                                            # rows 20 apart, beginning at the fourth
    out = qmm.moe_plan(l, 1)
    assert out[4].tolist() == [0] * 4 + [n] + [0] * 7 and out[3].tolist() == [0] * 5 + [4096 - 96] * 7 or n % 128
    assert out[4].tolist() == [0] * 4 + [n] + [0] * 7
    assert out[3].tolist() == [0] * 5 + [-(-n // 128) * 128] * 7
    assert T.equal(out[2][:, 0], T.arange(n, device="cuda", dtype=T.int32))
    again = qmm.moe_plan(l.contiguous().bfloat16(), 1, out=tuple(T.empty_like(t) for t in out))
    assert all(T.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("first", [1, 2, 3, 4])
@pytest.mark.parametrize("k", [3, 4, 8, 12])
@pytest.mark.parametrize("n", [5, 32, 33, 700])
def test_routing_in_slices_of_one_array(T, qmm, n, k, first):
    """Arrays of the routing need 4-byte alignment and no more: all five from one array, words that no call may touch between."""
    E, K = 20, 64
    g = T.Generator(device="cuda").manual_seed(n + k)
    l, x = T.randn(n, E, generator=g, device="cuda"), T.randn(n, K, generator=g, device="cuda")
    whole = T.full((3 * n * k + 2 * E + 64,), 0x5A5A5A5A, dtype=T.int32, device="cuda")
    out, at, free = [], first, T.ones(len(whole), dtype=T.bool, device="cuda")
    for shape in ((n, k), (n, k), (n, k), (E,), (E,)):
        size = int(np.prod(shape))
        out.append(whole[at:at + size].view(shape))
        free[at:at + size] = False
        at += size
        at += (first - at) % 4 + 4                               # each begins as far from a multiple of 16 bytes as the first
    assert all(t.data_ptr() % 16 == 4 * first % 16 for t in out)
    out[1] = out[1].view(T.float32)
    got = qmm.moe_plan(l, k, out=tuple(out))
    qmm.check()
    check_plan(got, plan_of(l.double().cpu().numpy(), k, True), E)
    assert bool((whole[free] == 0x5A5A5A5A).all())
    _, weights, places, starts, counts = got
    R = qmm.moe_rows(n, E, k)
    fresh = [t.clone() for t in got]
    w = qmm.mx4_quantize(T.randn(E, 24, K, generator=g, device="cuda"))
    ys, outs = [], []
    for _, weights, places, starts, counts in (got, fresh):
        y = T.zeros(R, 24, device="cuda")
        qmm.moe_gemm(*qmm.moe_quantize(x, places, R), *w, starts, counts, routed=n * k, out=y)
        qmm.moe_gemm(*qmm.moe_quantize(T.ones(R, K, device="cuda"), places, R, sorted=True), *w, starts, counts, routed=n * k)
        ys.append(y)
        outs.append(qmm.moe_combine(y, weights, places))
    qmm.check()
    assert T.equal(*ys) and T.equal(*outs) and bool((whole[free] == 0x5A5A5A5A).all())


@pytest.mark.parametrize("n,K,E,k", [(1, 32, 4, 1), (9, 160, 8, 3), (70, 1056, 5, 2), (300, 2048, 64, 8), (33, 4096 + 32, 9, 4)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_routed(T, qmm, n, K, E, k, dtype):
    rng = np.random.default_rng(n + K)
    x = T.from_numpy(spread(rng, n, K + 32)).cuda().to(getattr(T, dtype))[:, :K]
    l = rng.standard_normal((n, E)).astype(np.float32)
    l[rng.random((n, E)) < 0.3] = -np.inf
    _, _, places, _, _ = qmm.moe_plan(T.from_numpy(l).cuda(), k)
    R = qmm.moe_rows(n, E, k)
    codes = T.full((R, K // 8), 0x5A5A5A5A, dtype=T.int32, device="cuda")
    scales = T.full((qmm.mx4_scales_size(R, K),), 99, dtype=T.uint8, device="cuda")
    qmm.moe_quantize(x, places, R, out=(codes, scales))
    qmm.check()
    want, s = ref.quantize(x.float().cpu().numpy())
    p, c, got = places.cpu().numpy(), ref.unpack(codes.cpu().numpy()), scales.cpu().numpy()
    at, _ = ref.scale_at(R, K)
    every, _ = ref.scale_at(R, -(-K // 128) * 128)
    held = np.zeros(R, bool)
    for t in range(n):
        for r in p[t][p[t] >= 0]:
            held[r] = True
            good = np.repeat(s[t] != 255, 32)                    # (a NaN block's codes say nothing)
            assert np.array_equal(c[r][good], want[t][good])
            assert np.array_equal(got[at[r]], s[t]) and not got[every[r, K // 32:]].any()
    assert (codes[T.from_numpy(~held).cuda()] == 0x5A5A5A5A).all() and (got[every[~held]] == 99).all()


@pytest.mark.parametrize("n,K,E,k", [(1, 32, 4, 1), (9, 160, 8, 3), (70, 1056, 5, 2), (300, 2048, 64, 8)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_sorted(T, qmm, n, K, E, k, dtype):
    """Only the rows of the places: others are neither read (NaN there reaches nothing) nor written."""
    rng = np.random.default_rng(n + K)
    l = rng.standard_normal((n, E)).astype(np.float32)
    l[rng.random((n, E)) < 0.3] = -np.inf
    _, _, places, _, _ = qmm.moe_plan(T.from_numpy(l).cuda(), k)
    R = qmm.moe_rows(n, E, k)
    p = places.cpu().numpy()
    held = np.zeros(R, bool)
    held[p[p >= 0]] = True
    x = spread(rng, R, K)
    x[~held] = np.nan
    x = T.from_numpy(x).cuda().to(getattr(T, dtype))
    codes = T.full((R, K // 8), 0x5A5A5A5A, dtype=T.int32, device="cuda")
    scales = T.full((qmm.mx4_scales_size(R, K),), 99, dtype=T.uint8, device="cuda")
    qmm.moe_quantize(x, places, R, sorted=True, out=(codes, scales))
    qmm.check()
    want, s = ref.quantize(x.float().cpu().numpy()[held])
    at, _ = ref.scale_at(R, K)
    every, _ = ref.scale_at(R, -(-K // 128) * 128)
    got = scales.cpu().numpy()
    assert np.array_equal(got[at[held]], s) and (got[every[~held]] == 99).all() and not got[every[held][:, K // 32:]].any()
    good = np.repeat(s != 255, 32, axis=1)
    assert np.array_equal(ref.unpack(codes.cpu().numpy())[held][good], want[good])
    assert (codes[T.from_numpy(~held).cuda()] == 0x5A5A5A5A).all()
    with pytest.raises(ValueError):
        qmm.moe_quantize(x, places, R + 128, sorted=True)


def test_places_outside_are_skipped(T, qmm):
    x = T.ones(4, 64, device="cuda")
    places = T.tensor([[0, -1], [128, 3], [1 << 30, -(1 << 31)], [127, 1]], dtype=T.int32, device="cuda")
    codes, scales = T.zeros(129, 8, dtype=T.int32, device="cuda"), T.zeros(1025, dtype=T.uint8, device="cuda")
    qmm.moe_quantize(x, places, 128, out=(codes[:128], scales[:512]))
    y = qmm.mx4_dequant(codes[:128], scales[:512])
    assert sorted(y[:, 0].nonzero().flatten().tolist()) == [0, 1, 3, 127] and not codes[128].any() and not scales[512:].any()
    codes.zero_()
    qmm.moe_quantize(T.ones(128, 64, device="cuda"), places, 128, sorted=True, out=(codes[:128], scales[:512]))
    assert T.equal(y, qmm.mx4_dequant(codes[:128], scales[:512])) and not codes[128].any()
    out = qmm.moe_combine(y, T.full((4, 2), 2.0, device="cuda"), places)
    assert out[:, 5].tolist() == [2.0, 2.0, 0.0, 4.0]
    w = T.tensor([[1.0, float("nan")]] * 4, device="cuda")
    assert out.shape == (4, 64) and qmm.moe_combine(y, w, places)[0, 0] == 1.0


def experts_case(T, rng, counts, N, K, gated):
    E = len(counts)
    starts = np.concatenate(([0], np.cumsum((np.array(counts) + 127) // 128 * 128)[:-1]))
    R = int(starts[-1] + -(-counts[-1] // 128) * 128)
    xc, xs, xv = matrix(rng, max(R, 1), K)
    two = 2 if gated else 1
    ws = [matrix(rng, N, K, K ** -0.5) for _ in range(E * two)]
    w = [on_gpu(T, c, s, 255) for c, s, _ in ws]
    lead = (E, 2) if gated else (E,)
    codes = T.stack([a[0] for a in w]).view(*lead, N, K // 8)
    scales = T.stack([a[1] for a in w]).view(*lead, -1)
    values = np.stack([v for *_, v in ws]).reshape(*lead, N, K)
    i32 = lambda v: T.tensor(np.asarray(v), dtype=T.int32, device="cuda")
    return xc, xs, xv, codes, scales, values, i32(starts), i32(counts), starts, R


@pytest.mark.parametrize("counts,N,K", [([1], 1, 32), ([3, 0, 1], 130, 96), ([0, 0, 5, 0], 256, 512), ([8] * 9, 300, 1056),
                                        ([1, 1, 0, 1, 1, 0, 1, 1], 2048, 1408), ([129, 64, 65, 0, 300], 257, 288),
                                        ([700, 5, 128, 256], 128, 640), ([40] * 30, 200, 352), ([33, 17, 250, 1, 0, 90], 384, 2080), ([900, 0, 300, 1, 513], 2000, 2720),
                                        ([257, 640, 128], 1100, 2080)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gated", [False, True])
def test_experts(T, qmm, counts, N, K, dtype, gated):
    rng = np.random.default_rng(sum(counts) + N + K)
    xc, xs, xv, codes, scales, values, st, ct, starts, R = experts_case(T, rng, counts, N, K, gated)
    own = np.zeros(R, bool)
    for s, n in zip(starts, counts):
        own[s:s + n] = True
    xs[~own] = 255                                               # rows of no expert hold anything
    x = on_gpu(T, xc, xs)
    results = []
    for routed in (None, sum(counts), 1, 100000):                # only the launch's shape
        y = T.full((R, N), 7.0, dtype=getattr(T, dtype), device="cuda")
        assert qmm.moe_gemm(*x, codes, scales, st, ct, routed=routed, gated=gated, out=y) is y
        qmm.check()
        for e, (s, n) in enumerate(zip(starts, counts)):
            if n:
                want, bound = ref.product(xv[s:s + n], values[e], gated)
                check_product(y[s:s + n], want, bound, dtype)
        assert (y[T.from_numpy(~own).cuda()] == 7).all()


def test_experts_reach_pairs(qmm):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the rule counts SMs")
    R = 1024 + 384 + 128 + 640
    assert qmm.mx4_gemm_tile(R, 2000, 2720, experts=5, routed=1714) > 1024
    assert qmm.mx4_gemm_tile(R, 2000, 2720, gated=True, experts=5, routed=1714) > 1024
    assert qmm.mx4_gemm_tile(128 * 9, 300, 1056, experts=9, routed=72) == 64


def test_experts_that_share_rows_stay_inside(T, qmm):
    """Not allowed, but no reason to leave the arrays: every expert claims all rows."""
    rng = np.random.default_rng(8)
    xc, xs, xv, codes, scales, values, st, ct, _, R = experts_case(T, rng, [128] * 40, 130, 64, False)
    y = T.full((R + 1, 130), 7.0, device="cuda")
    qmm.moe_gemm(*on_gpu(T, xc, xs), codes, scales, T.zeros_like(st), T.full_like(ct, R), out=y[:R])
    qmm.check()
    assert (y[R] == 7).all() and T.isfinite(y).all()


def test_experts_with_bad_starts_and_counts(T, qmm):
    rng = np.random.default_rng(2)
    xc, xs, xv, codes, scales, values, st, ct, _, R = experts_case(T, rng, [100, 20, 30, 40, 50], 64, 64, False)
    assert R == 640
    st = T.tensor([0, 130, 1 << 30, -128, 512], dtype=T.int32, device="cuda")      # no multiple, past the end, negative
    ct = T.tensor([-5, 20, 30, 40, 1 << 30], dtype=T.int32, device="cuda")         # fewer than none; past the end
    y = T.full((R + 1, 64), 7.0, device="cuda")
    qmm.moe_gemm(*on_gpu(T, xc, xs), codes, scales, st, ct, out=y[:R])
    qmm.check()
    assert (y[:512] == 7).all() and (y[R] == 7).all()
    want, bound = ref.product(xv[512:], values[4])
    check_product(y[512:R], want, bound, "float32")


@pytest.mark.parametrize("n,k,N", [(1, 1, 1), (3, 2, 7), (8, 6, 2048), (50, 8, 1001), (130, 32, 24), (1000, 4, 516), (17, 3, 8200)])
@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("out_dtype", ["float32", "bfloat16"])
def test_combine(T, qmm, n, k, N, y_dtype, out_dtype):
    rng = np.random.default_rng(n + N)
    R = 128 * (1 + n * k // 128)
    y = T.from_numpy(rng.standard_normal((R, N))).to(getattr(T, y_dtype)).cuda()
    w = T.from_numpy(rng.random((n, k)).astype(np.float32)).cuda()
    p = rng.integers(-R // 4, R, (n, k))
    places = T.from_numpy(p.astype(np.int32)).cuda()
    out = qmm.moe_combine(y, w, places, dtype=getattr(T, out_dtype))
    ones = qmm.moe_combine(y, None, places, dtype=getattr(T, out_dtype))
    qmm.check()
    yv, wv = y.double().cpu().numpy(), w.double().cpu().numpy()
    half = 2.0 ** -8 if out_dtype == "bfloat16" else 2.0 ** -24
    for got, weights in ((out, wv), (ones, np.ones_like(wv))):
        rows = np.where((p >= 0)[..., None], yv[np.maximum(p, 0)], 0) * weights[..., None]
        want, size = rows.sum(1), np.abs(rows).sum(1)
        # a product and a sum each of k times
        assert (np.abs(got.double().cpu().numpy() - want) <= half * np.abs(want) + (k + 1) * 2.0 ** -24 * (1 + half) * size).all()


def layer(qmm, x, logits, k, w1, w2):
    """Tokens to their experts and back: what a user's program calls."""
    _, weights, places, starts, counts = qmm.moe_plan(logits, k)
    n, R = x.shape[0], qmm.moe_rows(*logits.shape, k)
    h = qmm.moe_gemm(*qmm.moe_quantize(x, places, R), *w1, starts, counts, routed=n * k, gated=True, dtype=x.dtype)
    y = qmm.moe_gemm(*qmm.moe_quantize(h, places, R, sorted=True), *w2, starts, counts, routed=n * k, dtype=x.dtype)
    return qmm.moe_combine(y, weights, places), h, y


@pytest.mark.parametrize("n,dtype", [(1, "float32"), (6, "float32"), (40, "bfloat16"), (333, "bfloat16")])
def test_whole_layer(T, qmm, n, dtype):
    """Every step against float64 of what the step before gave; then captured, and replayed with other tokens, on two streams."""
    K, F, E, k = 256, 160, 12, 3
    g = T.Generator(device="cuda").manual_seed(n)
    rand = lambda *s: T.randn(s, generator=g, device="cuda")
    w1, w2 = qmm.mx4_quantize(rand(E, 2, F, K) * K ** -0.5), qmm.mx4_quantize(rand(E, K, F) * F ** -0.5)
    v1, v2 = qmm.mx4_dequant(*w1).double().cpu().numpy(), qmm.mx4_dequant(*w2).double().cpu().numpy()

    def check(x, logits, out, h, y):
        experts, weights, places, starts, counts = plan_of(logits.double().cpu().numpy(), k, True)
        xq = ref.values(*ref.quantize(x.float().cpu().numpy()))
        hv, yv = h.float().cpu().numpy(), y.double().cpu().numpy()
        for e in range(E):
            s, c = starts[e], counts[e]
            if not c:
                continue
            rows = np.argsort(np.where(experts == e, places, 1 << 30).min(1), kind="stable")[:c]
            want, bound = ref.product(xq[rows], v1[e], True)
            check_product(h[s:s + c], want, bound, dtype)
            want, bound = ref.product(ref.values(*ref.quantize(hv[s:s + c])), v2[e])
            check_product(y[s:s + c], want, bound, dtype)
        want = (yv[places] * weights[..., None]).sum(1)
        half = 2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -24
        assert (np.abs(out.double().cpu().numpy() - want)
                <= half * np.abs(want) + (E + 20) * 2.0 ** -23 * (np.abs(yv[places]) * weights[..., None]).sum(1)).all()

    x, logits = rand(n, K).to(getattr(T, dtype)), rand(n, E)
    check(x, logits, *layer(qmm, x, logits, k, w1, w2))
    qmm.check()
    sets = []
    for _ in range(2):
        a, b = x.clone(), logits.clone()
        graph = T.cuda.CUDAGraph()
        with T.cuda.graph(graph):
            out = layer(qmm, a, b, k, w1, w2)
        sets.append((a, b, graph, out, T.cuda.Stream()))
    for _ in range(3):
        for a, b, graph, _, s in sets:
            a.copy_(rand(n, K))
            b.copy_(rand(n, E))
        T.cuda.synchronize()
        for a, b, graph, _, s in sets:
            with T.cuda.stream(s):
                graph.replay()
        T.cuda.synchronize()
        for a, b, _, out, _ in sets:
            check(a, b, *out)
    qmm.check()
