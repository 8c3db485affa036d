"""The microscaled 4-bit quantizer and product against float64."""
import numpy as np
import pytest

import mx4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_gb300 import build
    build.build()
    return torch


@pytest.fixture(scope="module")
def qmm(T):
    from quantized_weight_gb300 import qmm
    return qmm


def spread(rng, rows, K):
    """Values of many sizes: rows and columns of their own scale, exact borders, zeros of both signs, tiny and large blocks."""
    x = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1))) * np.exp(rng.standard_normal((1, K)))
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, -0.0, -2.5, -0.25], (rows, K))
    x = np.where(rng.random((rows, K)) < 0.2, border, x)
    power = np.where(rng.random((rows, K // 32)) < 0.2, rng.integers(-150, 125, (rows, K // 32)), 0)
    with np.errstate(over="ignore"):
        return (x.reshape(rows, -1, 32) * np.exp2(power)[..., None]).reshape(rows, K).astype(np.float32)


def check_quantized(codes, scales, x):
    want, s = ref.quantize(x)
    rows, K = x.shape
    at, size = ref.scale_at(rows, K)
    got = scales.cpu().numpy()
    assert got.shape == (size,)
    assert np.array_equal(got[at], s)
    good = np.repeat(s != 255, 32, axis=1)                       # (a NaN block's codes say nothing)
    assert np.array_equal(np.where(good, ref.unpack(codes.cpu().numpy()), 0), np.where(good, want, 0))
    every, _ = ref.scale_at(rows, -(-K // 128) * 128)
    assert not got[every[:, K // 32:]].any()                     # blocks past K


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 256), (31, 288), (33, 544), (127, 128), (128, 4096), (130, 1056),
                                    (257, 64), (8, 8192)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize(T, qmm, rows, K, dtype):
    x = T.from_numpy(spread(np.random.default_rng(rows * K), rows, K)).cuda().to(getattr(T, dtype))
    codes, scales = qmm.mx4_quantize(x)
    w = qmm.mx4_dequant(codes, scales)
    qmm.check()
    check_quantized(codes, scales, x.float().cpu().numpy())
    c, s = ref.quantize(x.float().cpu().numpy())
    w, want = w.cpu().numpy(), ref.values(c, s)                  # (a value beyond float32 is an infinity, its block NaN)
    assert np.array_equal(w.astype(np.float64), want, equal_nan=True)
    good = ~np.isnan(want)
    assert np.array_equal(np.signbit(w)[good], (c >= 8)[good])


def test_quantize_what_is_not_finite_and_extremes(T, qmm):
    x = np.ones((4, 160), np.float32)
    x[0, 5], x[0, 40], x[1, 70], x[2, 130] = np.nan, np.inf, -np.inf, np.float32(3.4028235e38)
    x[3, :32] = np.float32(1e-45)                                # the smallest subnormal
    x[3, 32:64] = 0.0
    x[3, 64:96] = np.float32(-2.0 ** -126)
    codes, scales = qmm.mx4_quantize(T.from_numpy(x).cuda())
    w = qmm.mx4_dequant(codes, scales).cpu().numpy()
    check_quantized(codes, scales, x)
    bad = np.isnan(w).reshape(4, 5, 32)
    assert bad.all(-1).sum() == 3 and bad.any(-1).sum() == 3 and bad[0, 0, 0] and bad[0, 1, 0] and bad[1, 2, 0]
    c, s = ref.quantize(x)
    good = ~np.isnan(w)
    assert np.array_equal(w[good].astype(np.float64), ref.values(c, s)[good])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_strides_matrices_and_outputs(T, qmm, dtype):
    rng = np.random.default_rng(3)
    full = T.from_numpy(spread(rng, 3 * 50, 256)).cuda().to(getattr(T, dtype)).view(3, 50, 256)
    x = full[:, 1:48:2, 32:224]                                  # rows of a stride, matrices of another
    out = (T.full((3, 24, 24), -1, dtype=T.int32, device="cuda"), T.full((3, 1024), 77, dtype=T.uint8, device="cuda"))
    codes, scales = qmm.mx4_quantize(x, out=out)
    assert codes is out[0] and scales is out[1]
    for i in range(3):
        check_quantized(codes[i], scales[i], x[i].float().cpu().numpy())
    w = qmm.mx4_dequant(codes, scales)
    for i in range(3):
        assert T.equal(w[i], qmm.mx4_dequant(codes[i], scales[i]))
    four = full.view(3, 2, 25, 256)
    c4, s4 = qmm.mx4_quantize(four)
    assert c4.shape == (3, 2, 25, 32) and s4.shape == (3, 2, 1024)
    check_quantized(c4[2, 1], s4[2, 1], four[2, 1].float().cpu().numpy())


def test_quantize_refusals(T, qmm):
    x = T.zeros(4, 64, device="cuda")
    for bad in (x[:, ::2], x[0], x.t()):
        with pytest.raises((ValueError, qmm.QmmError)):
            qmm.mx4_quantize(bad)
    with pytest.raises(qmm.QmmError):
        qmm.mx4_quantize(T.zeros(4, 66, device="cuda")[:, :64])          # rows at multiples of 8 bytes
    with pytest.raises(ValueError):
        qmm.mx4_quantize(T.zeros(4, 48, device="cuda"))
    with pytest.raises(ValueError):
        qmm.mx4_quantize(x, out=(T.zeros(4, 8, dtype=T.int32, device="cuda"), T.zeros(511, dtype=T.uint8, device="cuda")))
    assert qmm.mx4_quantize(x[:0])[0].shape == (0, 8)
    assert qmm.mx4_quantize(x[:, :0])[1].shape == (0,)


def test_dequant_every_scale_and_code(T, qmm):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    w = qmm.mx4_dequant(T.from_numpy(ref.pack(codes)).cuda(), T.from_numpy(ref.tiles(scales)).cuda()).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.values(codes, scales).astype(np.float32)              # 6 * 2 ** 127 is an infinity in float32
    assert np.array_equal(w, want, equal_nan=True)


def matrix(rng, rows, K, width=1.0):
    """(codes, scale bytes, float64 values) of a matrix whose blocks differ in size."""
    x = rng.standard_normal((rows, K)) * np.exp(0.7 * rng.standard_normal((rows, 1))) * width
    c, s = ref.quantize(x)
    return c, s, ref.values(c, s)


def on_gpu(T, c, s, fill=0):
    return T.from_numpy(ref.pack(c)).cuda(), T.from_numpy(ref.tiles(s, fill)).cuda()


def check_product(y, want, bound, dtype):
    got = y.float().cpu().numpy().astype(np.float64)
    half = 2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -24
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= (bound * (1 + half) + half * np.abs(want))[ok]).all()


SIZES = [(1, 1, 32), (1, 128, 64), (3, 130, 96), (8, 257, 256), (9, 64, 1056), (16, 1000, 512), (17, 129, 2080), (33, 384, 288),
         (64, 256, 4096), (65, 300, 320), (100, 128, 992), (127, 511, 256), (128, 128, 128), (129, 1, 384), (200, 640, 224),
         (256, 256, 1024), (257, 390, 160), (300, 2000, 96), (500, 129, 5120), (1024, 1025, 512), (2500, 300, 256)]


def test_every_kernel_is_reached(T, qmm):
    """By the sizes of this file and of the experts' tests, on a GB300."""
    if T.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the rule counts SMs")
    assert {qmm.mx4_gemm_tile(M, N, K) for M, N, K in SIZES + LARGE} == {64, 128, 192, 256, 256 + 1024}
    assert {qmm.mx4_gemm_tile(M, N, K, gated=True) for M, N, K in SIZES + LARGE} == {64, 128, 128 + 1024}


# the first two take pairs of CTAs (the second CTA without weight rows in the last tile, and tokens of one row), then gated
# ones, then wide tiles of one
LARGE = [(1500, 2900, 2720), (1281, 2900, 2592), (900, 1500, 2208), (641, 1300, 2080), (1281, 3000, 1024), (1000, 2900, 512)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gated", [False, True])
def test_large_product(T, qmm, M, N, K, dtype, gated):
    test_product(T, qmm, M, N, K, dtype, gated)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gated", [False, True])
def test_product(T, qmm, M, N, K, dtype, gated):
    rng = np.random.default_rng(M * 1000003 + N * 1009 + K)
    xc, xs, xv = matrix(rng, M, K)
    ws = [matrix(rng, N, K, K ** -0.5) for _ in range(2 if gated else 1)]
    # scales of rows past the last are never used, whatever they are
    x = on_gpu(T, xc, xs, 255)
    w = [on_gpu(T, c, s, 255) for c, s, _ in ws]
    codes, scales = (T.stack([a[0] for a in w]), T.stack([a[1] for a in w])) if gated else w[0]
    out = T.full((M + 1, N), 7.0, dtype=getattr(T, dtype), device="cuda")
    y = qmm.mx4_gemm(*x, codes, scales, gated=gated, out=out[:M])
    qmm.check()
    want, bound = ref.product(xv, np.stack([v for *_, v in ws]) if gated else ws[0][2], gated)
    check_product(y, want, bound, dtype)
    assert (out[M] == 7).all()
    assert T.equal(y, qmm.mx4_gemm(*x, codes, scales, gated=gated, dtype=getattr(T, dtype)))   # the same every time


def test_product_of_every_scale(T, qmm):
    """Powers of two far apart, sums exact: one block a row that is not zero."""
    rng = np.random.default_rng(5)
    M, N, K = 64, 96, 256
    c = np.zeros((M, K), np.uint8)
    s = rng.integers(0, 255, (M, K // 32)).astype(np.uint8)
    for m in range(M):
        c[m, 32 * (m % 8):32 * (m % 8) + 32] = rng.integers(0, 16, 32)
    s[np.arange(M), np.arange(M) % 8] = np.linspace(60, 190, M).astype(np.uint8)
    wc = rng.integers(0, 16, (N, K)).astype(np.uint8)
    w = rng.integers(120, 135, (N, K // 32)).astype(np.uint8)
    y = qmm.mx4_gemm(*on_gpu(T, c, s), *on_gpu(T, wc, w)).cpu().numpy().astype(np.float64)
    want, bound = ref.product(ref.values(c, s), ref.values(wc, w))
    assert (np.abs(y - want) <= bound).all()


@pytest.mark.parametrize("M,N,K", [(5, 200, 512), (130, 150, 288), (600, 256, 1024)])
def test_product_of_what_is_not_finite(T, qmm, M, N, K):
    """A NaN block reaches the results of its row and no others."""
    rng = np.random.default_rng(M)
    xc, xs, xv = matrix(rng, M, K)
    wc, ws, wv = matrix(rng, N, K)
    xs[M // 2, 1] = ws[7, -1] = ws[N - 1, 0] = 255
    xv, wv = ref.values(xc, xs), ref.values(wc, ws)
    y = qmm.mx4_gemm(*on_gpu(T, xc, xs), *on_gpu(T, wc, ws))
    qmm.check()
    want = np.where(np.isnan(xv).any(1)[:, None] | np.isnan(wv).any(1)[None], np.nan, 0.0)
    assert np.array_equal(np.isnan(y.cpu().numpy()), np.isnan(want))
    good_m, good_n = ~np.isnan(xv).any(1), ~np.isnan(wv).any(1)
    ok, bound = ref.product(xv[good_m], wv[good_n])
    assert (np.abs(y.cpu().numpy()[good_m][:, good_n] - ok) <= bound + 2.0 ** -24 * np.abs(ok)).all()


def test_gated_extremes(T, qmm):
    """silu far out: z below -88 gives -0 times u, not NaN."""
    N, K = 130, 32
    x = np.ones((3, K), np.float32)
    g = np.repeat(np.array([[-6.0], [-0.5], [0.0], [6.0]], np.float32), 33, 0)[:N] * np.ones((1, K), np.float32)
    u = np.full((N, K), 2.0, np.float32)
    y = qmm.mx4_gemm(*qmm.mx4_quantize(T.from_numpy(x).cuda()),
                     *qmm.mx4_quantize(T.from_numpy(np.stack((g, u))).cuda()), gated=True)
    want, bound = ref.product(x.astype(np.float64), np.stack((g, u)).astype(np.float64), True)
    assert (np.abs(y.cpu().numpy() - want) <= bound + 2.0 ** -24 * np.abs(want)).all()


# single CTAs of 64 tokens, K in parts over a cluster, 128 tokens, pairs
@pytest.mark.parametrize("M,N,K", [(3, 400, 32), (8, 400, 4096), (300, 400, 512), (1500, 2900, 2720)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gated_far_out(T, qmm, M, N, K, dtype):
    """silu where exp(-z) nears the end of float32 and passes it, times a u that makes a whole result of it."""
    v = np.arange(N) % 360 / 2                                   # -z, 0 to 179.5
    g, u = np.zeros((N, K)), np.zeros((N, K))
    full = (v // 6).astype(int)
    rest = v - 6 * full                                          # of halves, as two values of the format
    top = np.array([0, 0.5, 1, 1.5, 2, 2, 3, 3, 4, 4, 4, 4])[(2 * rest).astype(int)]
    for n in range(N):
        g[n, :full[n]] = -6
        g[n, 30], g[n, 31] = -top[n], -(rest[n] - top[n])
    u[:, 0] = np.where(v < 60, -1.5, 1.5 * 2.0 ** 120)
    x = np.ones((M, K))
    made = [ref.quantize(a) for a in (x, g, u)]
    assert all(np.array_equal(ref.values(*m), a) for m, a in zip(made, (x, g, u)))
    w = [on_gpu(T, *m) for m in made[1:]]
    y = qmm.mx4_gemm(*on_gpu(T, *made[0]), T.stack([a[0] for a in w]), T.stack([a[1] for a in w]), gated=True, dtype=getattr(T, dtype))
    qmm.check()
    want = (-v / (1 + np.exp(v)) * u[:, 0])[None]
    got = y.double().cpu().numpy()
    # Both sums are exact.  float32: an exponential of 2 ulp, taken twice far out, and a quotient of 1 ulp, four roundings: 16
    # halves of an ulp at most.  bfloat16: the quick exponential, 2^-22 and |z| * 2^-23 where it is used (z from -64 up), less
    # than 2^-16.9 with the others, and one rounding to 8 bits.  Far below what is normal a result has fewer bits.
    each = 2.0 ** -20 if dtype == "float32" else 2.0 ** -16.8 + 2.0 ** -8
    assert (np.abs(got - want) <= each * np.abs(want) + 2.0 ** -126).all()
    assert (np.abs(want) > 1e-6)[0, (v > 85) & (v < 95)].all()   # (whole results among them)


def test_product_refusals(T, qmm):
    x = qmm.mx4_quantize(T.ones(4, 64, device="cuda"))
    w = qmm.mx4_quantize(T.ones(6, 64, device="cuda"))
    other = qmm.mx4_quantize(T.ones(6, 96, device="cuda"))
    for args, kw in (((*x, *other), {}), ((*x, *w), dict(gated=True)), ((*x, w[0], other[1][:511]), {}),
                     ((*x, w[0].float(), w[1]), {}), ((*x, *w), dict(out=T.empty(4, 5, device="cuda"))),
                     ((*x, *w), dict(dtype=T.float16)), ((x[0].t().contiguous().t(), x[1], *w), {})):
        with pytest.raises((ValueError, TypeError)):
            qmm.mx4_gemm(*args, **kw)
    assert qmm.mx4_gemm(*qmm.mx4_quantize(T.ones(0, 64, device="cuda")), *w).shape == (0, 6)


def test_product_on_another_stream_and_in_graphs(T, qmm):
    """Two streams at once and captured calls: no call keeps anything between calls."""
    rng = np.random.default_rng(11)
    mats = [(matrix(rng, 8, 1024), matrix(rng, 640, 1024)) for _ in range(4)]
    dev = [(on_gpu(T, *x[:2]), on_gpu(T, *w[:2])) for x, w in mats]
    plain = [qmm.mx4_gemm(*x, *w) for x, w in dev]
    streams = [T.cuda.Stream() for _ in range(2)]
    T.cuda.synchronize()
    for _ in range(20):
        got = [qmm.mx4_gemm(*x, *w, stream=streams[i % 2]) for i, (x, w) in enumerate(dev)]
    T.cuda.synchronize()
    assert all(T.equal(a, b) for a, b in zip(got, plain))
    graphs, outs = [], []
    for x, w in dev[:2]:
        g = T.cuda.CUDAGraph()
        with T.cuda.graph(g):
            outs.append(qmm.mx4_gemm(*x, *w))
        graphs.append(g)
    for a, b in zip(dev[0][0], dev[2][0]):
        a.copy_(b)                                               # the first graph gets the third product's x
    for s, g in zip(streams, graphs):
        s.wait_stream(T.cuda.current_stream())
        with T.cuda.stream(s):
            g.replay()
    T.cuda.synchronize()
    want, bound = ref.product(mats[2][0][2], mats[0][1][2])
    check_product(outs[0], want, bound, "float32")
    assert T.equal(outs[1], plain[1])
