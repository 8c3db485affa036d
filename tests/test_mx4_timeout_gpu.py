"""A bounded wait of the microscaled product that runs out, on the GPU, without faulting or hanging it: the test hook makes the
epilogue of every block wait on a barrier that nothing completes, while copies and products are in flight.  All roles have to
leave, nothing is written, the launch is reported once, and the next call is right."""
import time

import numpy as np
import pytest

import mx4_reference as ref
from test_mx4_gpu import T, check_product, matrix, on_gpu, qmm  # noqa: F401

pytestmark = pytest.mark.gpu

TIMEOUT = -6


def fails_once_then_is_right(T, qmm, call, out, check):
    T.cuda.synchronize()
    qmm.check()
    qmm.test_timeout_next_mx4(200_000)
    call()
    with pytest.raises(qmm.QmmError) as e:
        qmm.check()
    assert e.value.status == TIMEOUT
    qmm.check()                                                  # reported once
    assert bool((out == 7.0).all())
    for _ in range(2):                                           # the hook was taken by one launch only
        call()
    qmm.check()
    check()


# K in parts over a cluster; one item a block and several, by one CTA and by pairs; rings longer and shorter than K
@pytest.mark.parametrize("M,N,K", [(8, 256, 4096), (3, 130, 96), (100, 20000, 512), (1000, 2900, 512), (1281, 3000, 1024),
                                   (1500, 2900, 2720), (3000, 5000, 2048)])
@pytest.mark.parametrize("gated", [False, True])
def test_wait_runs_out(T, qmm, M, N, K, gated):
    rng = np.random.default_rng(M)
    xc, xs, xv = matrix(rng, M, K)
    ws = [matrix(rng, N, K, K ** -0.5) for _ in range(2 if gated else 1)]
    w = [on_gpu(T, c, s) for c, s, _ in ws]
    codes, scales = (T.stack([a[0] for a in w]), T.stack([a[1] for a in w])) if gated else w[0]
    x = on_gpu(T, xc, xs)
    out = T.full((M, N), 7.0, device="cuda")
    some = rng.integers(0, M, 40)

    def check():
        want, bound = ref.product(xv[some], np.stack([v for *_, v in ws]) if gated else ws[0][2], gated)
        check_product(out[T.from_numpy(some).cuda()], want, bound, "float32")
    fails_once_then_is_right(T, qmm, lambda: qmm.mx4_gemm(*x, codes, scales, gated=gated, out=out), out, check)


# (under the hook one CTA of each pair copies nothing, the first or the second by turns, while the other fills its ring)
@pytest.mark.parametrize("M,N,K", [(1500, 2900, 2720), (1281, 2900, 2592), (2500, 5000, 2720)])
@pytest.mark.parametrize("gated", [False, True])
def test_pairs_know_of_each_others_copies(T, qmm, M, N, K, gated):
    """Copies that only one CTA of a pair has begun are waited for by what has landed: at once, not until a limit of 2 s."""
    if T.cuda.get_device_properties(0).multi_processor_count == 152:
        assert qmm.mx4_gemm_tile(M, N, K, gated=gated) > 1024
    x = T.randn(M, K, device="cuda")
    w = T.randn(*((2, N, K) if gated else (N, K)), device="cuda") * K ** -0.5
    x, w = qmm.mx4_quantize(x), qmm.mx4_quantize(w)
    want = qmm.mx4_gemm(*x, *w, gated=gated)
    qmm.check()
    out = T.full((M, N), 7.0, device="cuda")
    for limit in (50_000, 200_000):
        begin = time.monotonic()
        qmm.test_timeout_next_mx4(limit)
        qmm.mx4_gemm(*x, *w, gated=gated, out=out)
        with pytest.raises(qmm.QmmError) as e:
            qmm.check()
        assert time.monotonic() - begin < 1.0
        assert e.value.status == TIMEOUT and bool((out == 7.0).all())
    again = qmm.mx4_gemm(*x, *w, gated=gated)
    qmm.check()
    assert T.equal(again, want)


def test_wait_runs_out_among_experts(T, qmm):
    rng = np.random.default_rng(1)
    E, N, K, n = 12, 300, 544, 40
    xc, xs, xv = matrix(rng, 128 * E, K)
    ws = [matrix(rng, N, K, K ** -0.5) for _ in range(E)]
    w = [on_gpu(T, c, s) for c, s, _ in ws]
    codes, scales, x = T.stack([a[0] for a in w]), T.stack([a[1] for a in w]), on_gpu(T, xc, xs)
    starts = T.arange(E, dtype=T.int32, device="cuda") * 128
    counts = T.full((E,), n, dtype=T.int32, device="cuda")
    out = T.full((128 * E, N), 7.0, device="cuda")

    def check():
        for e in range(E):
            want, bound = ref.product(xv[128 * e:128 * e + n], ws[e][2])
            check_product(out[128 * e:128 * e + n], want, bound, "float32")
    fails_once_then_is_right(T, qmm, lambda: qmm.moe_gemm(*x, codes, scales, starts, counts, out=out), out, check)


def test_limits_of_the_hook(qmm):
    for limit in (10, 10 ** 9):
        with pytest.raises(qmm.QmmError):
            qmm.test_timeout_next_mx4(limit)
