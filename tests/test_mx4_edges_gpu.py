"""Microscaled products and routing where sizes pass a border: past 4 GiB, past what a CTA lists or sorts at once, many experts,
no tokens; and calls beside one another."""
import numpy as np
import pytest

import mx4_reference as ref
from test_mx4_gpu import T, check_product, matrix, on_gpu, qmm  # noqa: F401

pytestmark = pytest.mark.gpu


def room(T, gigabytes):
    T.cuda.empty_cache()
    if T.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip("not enough free memory")


@pytest.mark.parametrize("M,N,K", [(66000, 17000, 64), (20000, 8200, 32)])
def test_product_of_many_items(T, qmm, M, N, K):
    """An output past 4 GiB, and more items than a CTA lists before it begins."""
    room(T, 20)
    rng = np.random.default_rng(M)
    xc, xs, xv = matrix(rng, M, K)
    wc, ws, wv = matrix(rng, N, K, K ** -0.5)
    y = qmm.mx4_gemm(*on_gpu(T, xc, xs), *on_gpu(T, wc, ws))
    qmm.check()
    some = np.r_[0, M - 1, rng.integers(0, M, 60)]
    want, bound = ref.product(xv[some], wv)
    check_product(y[T.from_numpy(some).cuda()], want, bound, "float32")


def test_quantize_past_4_gib(T, qmm):
    room(T, 30)
    rows, K = 70000, 65536                               # 9 GB of bfloat16, past 2^32 elements
    x = T.zeros(rows, K, dtype=T.bfloat16, device="cuda")
    last = T.randn(130, K, device="cuda").bfloat16()
    x[-130:] = last
    codes, scales = qmm.mx4_quantize(x)
    c, s = ref.quantize(last.float().cpu().numpy())
    assert np.array_equal(ref.unpack(codes[-130:].cpu().numpy()), c)
    at, _ = ref.scale_at(130 + 128, K)
    first = (rows - 130) // 128                          # the scale tiles of the last rows
    tiles = scales.view(-1, K // 128 * 512)[first:].flatten().cpu().numpy()
    assert np.array_equal(tiles[at[(rows - 130) % 128:][:130]], s)
    assert not codes[:-130].any()


def test_dequant_past_31_bits_of_words(T, qmm):
    room(T, 100)
    K, rows = 1 << 15, (1 << 19) + 130                   # 17 G elements: more than one launch
    codes = T.zeros(rows, K // 8, dtype=T.int32, device="cuda")
    codes[-130:] = T.randint(-2 ** 31, 2 ** 31 - 1, (130, K // 8), device="cuda", dtype=T.int32)
    codes[:2] = codes[-2:]
    scales = T.full((qmm.mx4_scales_size(rows, K),), 128, dtype=T.uint8, device="cuda")
    w = qmm.mx4_dequant(codes, scales)
    want = ref.values(ref.unpack(codes[-130:].cpu().numpy()), np.full((130, K // 32), 128, np.uint8))
    assert np.array_equal(w[-130:].double().cpu().numpy(), want)
    assert T.equal(w[:2], w[-2:]) and not w[2:-130:1000].any()
    del w, codes, scales
    T.cuda.empty_cache()


@pytest.mark.parametrize("n,E,k", [(40000, 40, 3), (20000, 1024, 2), (70001, 256, 1), (33, 1024, 32), (300, 700, 9)])
def test_plan_of_many(T, qmm, n, E, k):
    """More tokens than a CTA of the sort holds words for at once."""
    rng = np.random.default_rng(n)
    l = (rng.standard_normal((n, E)) + rng.standard_normal(E)).astype(np.float32)
    l[rng.random((n, E)) < 0.05] = -np.inf
    experts, weights, places, starts, counts = (t.cpu().numpy() for t in qmm.moe_plan(T.from_numpy(l).cuda(), k))
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    order = np.where(np.take_along_axis(l, order, 1) == -np.inf, -1, order)
    assert np.array_equal(experts, order)
    flat = order.flatten()
    want = np.bincount(flat[flat >= 0], minlength=E)
    assert np.array_equal(counts, want)
    assert np.array_equal(starts, np.concatenate(([0], np.cumsum((want + 127) // 128 * 128)[:-1])))
    by = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:want.sum()]
    rank = np.arange(want.sum()) - np.repeat(np.cumsum(want) - want, want)
    place = np.full(n * k, -1)
    place[by] = starts[flat[by]] + rank
    assert np.array_equal(places.flatten(), place)
    v = np.where(order >= 0, np.take_along_axis(l, np.maximum(order, 0), 1), -np.inf).astype(np.float64)
    p = np.exp(v - v[:, :1])
    assert np.allclose(weights, p / p.sum(1, keepdims=True), rtol=(8 + k / 2) * 2.0 ** -23, atol=2.0 ** -126)


@pytest.mark.parametrize("gated", [False, True])
def test_a_thousand_experts(T, qmm, gated):
    rng = np.random.default_rng(3)
    E, N, K = 1024, 40, 64
    counts = rng.choice([0, 0, 1, 3, 20], E)
    starts = np.concatenate(([0], np.cumsum((counts + 127) // 128 * 128)[:-1])).astype(np.int32)
    R = int(starts[-1] + 128)
    xc, xs, xv = matrix(rng, R, K)
    two = 2 if gated else 1
    wc, ws, wv = matrix(rng, E * two * N, K)
    codes = T.from_numpy(ref.pack(wc)).cuda().view(*((E, 2) if gated else (E,)), N, K // 8)
    scales = qmm.mx4_scales(T.from_numpy(ws.reshape(*((E, 2) if gated else (E,)), N, K // 32)).cuda())
    i32 = lambda a: T.from_numpy(a.astype(np.int32)).cuda()
    y = T.full((R, N), 7.0, device="cuda")
    qmm.moe_gemm(*on_gpu(T, xc, xs), codes, scales, i32(starts), i32(counts), routed=int(counts.sum()), gated=gated, out=y)
    qmm.check()
    wv = wv.reshape(E, two, N, K)
    held = np.zeros(R, bool)
    for e in np.flatnonzero(counts):
        s = slice(starts[e], starts[e] + counts[e])
        held[s] = True
        want, bound = ref.product(xv[s], wv[e] if gated else wv[e, 0], gated)
        check_product(y[s], want, bound, "float32")
    assert (y[T.from_numpy(~held).cuda()] == 7).all()


def test_no_tokens(T, qmm):
    E, k, K, N = 6, 2, 64, 40
    experts, weights, places, starts, counts = qmm.moe_plan(T.zeros(0, E, device="cuda"), k)
    assert not starts.any() and not counts.any() and places.shape == (0, k)
    R = qmm.moe_rows(0, E, k)
    w = qmm.mx4_quantize(T.ones(E, N, K, device="cuda"))
    y = qmm.moe_gemm(*qmm.moe_quantize(T.zeros(0, K, device="cuda"), places, R), *w, starts, counts, routed=0)
    assert y.shape == (0, N) and qmm.moe_combine(y, weights, places).shape == (0, N)
    # tokens of which none has an expert
    experts, weights, places, starts, counts = qmm.moe_plan(T.full((5, E), -float("inf"), device="cuda"), k)
    R = qmm.moe_rows(5, E, k)
    y = qmm.moe_gemm(*qmm.moe_quantize(T.ones(5, K, device="cuda"), places, R), *w, starts, counts, routed=10,
                     out=T.full((R, N), 7.0, device="cuda"))
    assert (y == 7).all() and not qmm.moe_combine(y, weights, places).any()
    qmm.check()


def test_calls_beside_one_another(T, qmm):
    """Pairs of CTAs, clusters that split K and single CTAs on three streams at once, and the plan's cluster beside them."""
    rng = np.random.default_rng(4)
    sizes = [(1500, 2900, 2720), (8, 512, 4096), (300, 700, 512)]
    mats = [(matrix(rng, M, K), matrix(rng, N, K)) for M, N, K in sizes]
    dev = [(on_gpu(T, *x[:2]), on_gpu(T, *w[:2])) for x, w in mats]
    alone = [qmm.mx4_gemm(*x, *w) for x, w in dev]
    l = T.randn(5000, 64, device="cuda")
    plan = qmm.moe_plan(l, 4)
    streams = [T.cuda.Stream() for _ in range(4)]
    T.cuda.synchronize()
    for _ in range(15):
        got = [qmm.mx4_gemm(*x, *w, stream=s) for s, (x, w) in zip(streams, dev)]
        again = qmm.moe_plan(l, 4, stream=streams[3])
    T.cuda.synchronize()
    qmm.check()
    assert all(T.equal(a, b) for a, b in zip(got, alone)) and all(T.equal(a, b) for a, b in zip(again, plan))


def test_calls_one_after_another(T, qmm):
    """Each may begin while the one before it ends, beside it on an SM, whatever tensor memory both want: clusters, two CTAs an
    SM, single ones and pairs in turns, also by a graph."""
    g = T.Generator(device="cuda").manual_seed(1)
    make = lambda *s: qmm.mx4_quantize(T.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5)
    sizes = [(8, 512, 4096, 1), (8, 512, 4096, 0), (8, 20000, 512, 0), (8, 20000, 512, 1), (100, 900, 512, 1), (1500, 2900, 2720, 0),
             (300, 700, 512, 0), (1500, 2900, 2720, 1), (1, 128, 64, 0), (1, 128, 64, 1)]
    calls = [(make(M, K), make(*((2, N, K) if gated else (N, K))), bool(gated)) for M, N, K, gated in sizes]
    alone = []
    for x, w, gated in calls:
        alone.append(qmm.mx4_gemm(*x, *w, gated=gated))
        T.cuda.synchronize()
    order = [i for step in (1, 3, 7, 9) for i in (step * j % len(calls) for j in range(len(calls)))]
    outs = [T.empty_like(alone[i]) for i in order]
    graph = T.cuda.CUDAGraph()
    with T.cuda.graph(graph):
        for i, out in zip(order, outs):
            x, w, gated = calls[i]
            qmm.mx4_gemm(*x, *w, gated=gated, out=out)
    for turn in range(6):
        for out in outs:
            out.fill_(7.0)
        if turn % 2:
            graph.replay()
        else:
            for i, out in zip(order, outs):
                x, w, gated = calls[i]
                qmm.mx4_gemm(*x, *w, gated=gated, out=out)
        qmm.check()
        assert all(T.equal(out, alone[i]) for i, out in zip(order, outs))


def test_weights_written_right_before(T, qmm):
    """A product may follow the quantizer of its weights at once, whatever begins early."""
    g = T.Generator(device="cuda").manual_seed(0)
    x = qmm.mx4_quantize(T.randn(8, 4096, generator=g, device="cuda"))
    ws = [T.randn(4096, 4096, generator=g, device="cuda") for _ in range(4)]
    want = []
    for w in ws:
        m = qmm.mx4_quantize(w)
        T.cuda.synchronize()
        want.append(qmm.mx4_gemm(*x, *m))
    m = tuple(T.empty_like(t) for t in m)
    y = [T.empty(8, 4096, device="cuda") for _ in ws]
    T.cuda.synchronize()
    for _ in range(10):
        for w, out in zip(ws, y):
            qmm.mx4_quantize(w, out=m)
            qmm.mx4_gemm(*x, *m, out=out)
        T.cuda.synchronize()
        assert all(T.equal(a, b) for a, b in zip(y, want))


def test_the_current_device(T, qmm, monkeypatch):
    x = qmm.mx4_quantize(T.ones(4, 64, device="cuda"))
    i = T.zeros(4, 2, dtype=T.int32, device="cuda")
    monkeypatch.setattr(qmm, "_device", lambda: 1)
    for call in (lambda: qmm.mx4_quantize(T.ones(4, 64, device="cuda:0")), lambda: qmm.mx4_gemm(*x, *x), lambda: qmm.mx4_dequant(*x),
                 lambda: qmm.moe_plan(T.ones(4, 8, device="cuda:0"), 2), lambda: qmm.moe_combine(T.ones(4, 8, device="cuda:0"), None, i)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_leading_dimensions_that_are_not_one_after_the_other(T, qmm):
    with pytest.raises(ValueError):
        qmm.mx4_quantize(T.ones(4, 3, 2, 64, device="cuda").transpose(0, 1))
