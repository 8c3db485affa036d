"""Refusals and limits of the microscaled 4-bit operators and of the routing to experts, without a GPU: no call here reaches
a kernel.  A size on the right side of a limit is shown by the refusal that comes after it (a missing pointer)."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from quantized_weight_gb300 import build as qbuild
from quantized_weight_gb300 import qmm

OK, ARG, SHAPE, ALIGN, UNSUP = 0, -1, -2, -3, -4
FAKE, MIS, ODD = 0x10000, 0x10004, 0x10002          # never dereferenced
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qmm.lib()


def quantize(L, x=FAKE, dtype=0, xm=0, xr=64, c=FAKE, s=FAKE, n=1, rows=4, K=64):
    return L.qmm_mx4_quantize(x, dtype, xm, xr, c, s, n, rows, K, None)


def dequant(L, c=FAKE, s=FAKE, w=FAKE, n=1, rows=4, K=64):
    return L.qmm_mx4_dequant(c, s, w, n, rows, K, None)


def gemm(L, x=FAKE, xs=FAKE, c=FAKE, s=FAKE, y=FAKE, dtype=0, gated=0, M=4, N=4, K=64):
    return L.qmm_mx4_gemm(x, xs, c, s, y, dtype, gated, M, N, K, None)


def plan(L, l=FAKE, dtype=0, stride=8, T=4, E=8, k=2, e=FAKE, w=FAKE, p=FAKE, st=FAKE, n=FAKE):
    return L.qmm_moe_plan(l, dtype, stride, T, E, k, 1, e, w, p, st, n, None)


def routed(L, x=FAKE, dtype=0, xr=64, p=FAKE, c=FAKE, s=FAKE, T=4, k=2, R=128, K=64, sorted=0):
    return L.qmm_moe_quantize(x, dtype, xr, sorted, p, c, s, T, k, R, K, None)


def experts(L, x=FAKE, xs=FAKE, c=FAKE, s=FAKE, st=FAKE, n=FAKE, y=FAKE, dtype=0, gated=0, m=8, R=128, E=4, N=4, K=64):
    return L.qmm_moe_gemm(x, xs, c, s, st, n, y, dtype, gated, m, R, E, N, K, None)


def combine(L, y=FAKE, yt=0, w=FAKE, p=FAKE, o=FAKE, ot=0, T=4, k=2, R=128, N=8):
    return L.qmm_moe_combine(y, yt, w, p, o, ot, T, k, R, N, None)


def test_quantize(L):
    for f in (quantize, routed):
        assert f(L, dtype=2) == UNSUP
        assert f(L, K=48) == SHAPE and f(L, K=-32) == SHAPE and f(L, K=BIG) == SHAPE
        assert f(L, x=None) == ARG and f(L, c=None) == ARG and f(L, s=None) == ARG
        assert f(L, x=MIS) == ALIGN and f(L, c=MIS) == ALIGN and f(L, s=MIS) == ALIGN
        assert f(L, xr=66) == ALIGN and f(L, xr=68, x=None) == ARG
        assert f(L, dtype=1, xr=68) == ALIGN and f(L, dtype=1, xr=72, x=None) == ARG
        assert f(L, K=0) == OK
    assert quantize(L, xm=2) == ALIGN
    assert quantize(L, rows=0) == OK and quantize(L, n=0) == OK and quantize(L, rows=-1) == SHAPE and quantize(L, n=-1) == SHAPE
    assert quantize(L, n=1 << 16, rows=1 << 15) == SHAPE and quantize(L, n=1 << 16, rows=(1 << 15) - 1, x=None) == ARG
    assert quantize(L, n=3, rows=715827882, x=None) == ARG and quantize(L, n=3, rows=715827883) == SHAPE
    assert routed(L, T=0) == OK and routed(L, R=0) == OK and routed(L, T=-1) == SHAPE and routed(L, R=BIG) == SHAPE
    assert routed(L, k=0) == SHAPE and routed(L, k=33) == SHAPE and routed(L, k=32, x=None) == ARG
    assert routed(L, T=1 << 30, k=2) == SHAPE and routed(L, T=(1 << 30) - 1, k=2, sorted=1, x=None) == ARG
    assert routed(L, p=None) == ARG and routed(L, p=ODD) == ALIGN and routed(L, p=MIS, x=None) == ARG


def test_dequant(L):
    assert dequant(L, K=40) == SHAPE and dequant(L, rows=BIG) == SHAPE and dequant(L, n=2, rows=1 << 30) == SHAPE
    for name in ("c", "s", "w"):
        assert dequant(L, **{name: None}) == ARG and dequant(L, **{name: MIS}) == ALIGN
    assert dequant(L, rows=0) == OK and dequant(L, K=0) == OK and dequant(L, n=0) == OK


def test_gemm(L):
    assert gemm(L, dtype=7) == UNSUP
    assert gemm(L, K=0) == SHAPE and gemm(L, K=33) == SHAPE and gemm(L, M=-1) == SHAPE and gemm(L, N=BIG) == SHAPE
    assert gemm(L, N=1 << 30, x=None) == ARG and gemm(L, N=1 << 30, gated=1) == SHAPE     # two matrices
    assert gemm(L, M=BIG - 1, N=63 * 128, x=None) == ARG and gemm(L, M=BIG - 1, N=64 * 128) == SHAPE     # tiles in 32 bits
    for name in ("x", "xs", "c", "s", "y"):
        assert gemm(L, **{name: None}) == ARG and gemm(L, **{name: MIS}) == ALIGN
    assert gemm(L, M=0) == OK and gemm(L, N=0) == OK


def test_experts(L):
    assert experts(L, dtype=-1) == UNSUP
    assert experts(L, E=0) == SHAPE and experts(L, E=1025) == SHAPE and experts(L, E=1024, x=None) == ARG
    assert experts(L, K=0) == SHAPE and experts(L, K=63) == SHAPE and experts(L, R=-1) == SHAPE and experts(L, m=-1) == SHAPE
    assert experts(L, E=64, N=1 << 25) == SHAPE and experts(L, E=63, N=1 << 25, x=None) == ARG
    assert experts(L, E=32, N=1 << 25, gated=1) == SHAPE
    for name in ("x", "xs", "c", "s", "y"):
        assert experts(L, **{name: None}) == ARG and experts(L, **{name: MIS}) == ALIGN
    for name in ("st", "n"):
        assert experts(L, **{name: None}) == ARG and experts(L, **{name: ODD}) == ALIGN
    assert experts(L, R=BIG - 1, N=63 * 128, x=None) == ARG and experts(L, R=BIG - 1, N=64 * 128) == SHAPE
    assert experts(L, R=0) == OK and experts(L, N=0) == OK


def test_gemm_tile(L):
    tile = L.qmm_mx4_gemm_tile
    assert tile(0, 0, 8, 0, 4096, 4096) == 64 and tile(0, 0, 8192, 0, 8192, 8192) == 256 + 1024
    assert tile(1, 48, 6144, 64, 1408, 2048) == 64
    for bad in ((0, 0, 8, 0, 64, 0), (0, 0, -1, 0, 64, 64), (0, 0, 8, -1, 64, 64), (0, 0, 8, 1025, 64, 64), (0, -1, 8, 4, 64, 64),
                (0, 0, 8, 64, 1 << 25, 64), (1, 0, 8, 0, 1 << 30, 64), (0, 0, BIG - 1, 0, 64 * 128, 64)):
        assert tile(*bad) == SHAPE
    with pytest.raises(qmm.QmmError):
        qmm.mx4_gemm_tile(8, 64, 48)


def test_plan(L):
    assert plan(L, dtype=3) == UNSUP
    assert plan(L, T=-1) == SHAPE and plan(L, E=0) == SHAPE and plan(L, E=1025) == SHAPE and plan(L, E=1024, l=None) == ARG
    assert plan(L, k=0) == SHAPE and plan(L, k=9) == SHAPE and plan(L, E=64, k=33) == SHAPE and plan(L, E=64, k=32, l=None) == ARG
    most = (BIG - 1 - 127 * 8) // 2
    assert plan(L, T=most, l=None) == ARG and plan(L, T=most + 1) == SHAPE
    for name in ("l", "e", "w", "p", "st", "n"):
        assert plan(L, **{name: None}) == ARG and plan(L, **{name: ODD}) == ALIGN
    assert plan(L, l=ODD, dtype=1, e=None) == ARG            # bfloat16 logits need two bytes' alignment
    assert plan(L, l=0x10001, dtype=1) == ALIGN


def test_combine(L):
    assert combine(L, yt=2) == UNSUP and combine(L, ot=2) == UNSUP
    assert combine(L, T=-1) == SHAPE and combine(L, k=0) == SHAPE and combine(L, k=33) == SHAPE and combine(L, R=-1) == SHAPE
    assert combine(L, N=BIG) == SHAPE
    assert combine(L, y=None) == ARG and combine(L, p=None) == ARG and combine(L, o=None) == ARG
    assert combine(L, y=MIS) == ALIGN and combine(L, o=MIS) == ALIGN and combine(L, p=ODD) == ALIGN and combine(L, w=ODD) == ALIGN
    assert combine(L, T=0) == OK and combine(L, N=0) == OK


def test_sizes(L):
    for rows, K in ((1, 32), (128, 128), (129, 160), (1000, 4096)):
        assert L.qmm_mx4_scales_size(rows, K) == ref.scale_at(rows, K)[1] == qmm.mx4_scales_size(rows, K)
    assert L.qmm_mx4_scales_size(-1, 32) == 0 and L.qmm_mx4_scales_size(4, 48) == 0 and L.qmm_mx4_scales_size(BIG, 32) == 0
    assert qmm.mx4_scales_size(0, 64) == 0
    for bad in ((-1, 32), (4, 48), (BIG, 32)):
        with pytest.raises(ValueError):
            qmm.mx4_scales_size(*bad)
    # T * k rows in at most min(E, T * k) experts
    assert L.qmm_moe_rows(1, 64, 1) == 128 and L.qmm_moe_rows(8, 64, 6) == 48 * 128
    assert L.qmm_moe_rows(1000, 4, 2) == 2560 and L.qmm_moe_rows(0, 4, 2) == 0
    for bad in ((-1, 4, 2), (4, 0, 1), (4, 4, 5), (4, 1025, 2), (1 << 30, 64, 4)):
        assert L.qmm_moe_rows(*bad) == -1
        with pytest.raises(ValueError):
            qmm.moe_rows(*bad)


@pytest.mark.parametrize("rows,blocks", [(1, 1), (128, 4), (33, 5), (300, 9)])
def test_scales_of_a_checkpoint(rows, blocks):
    plain = torch.arange(2 * rows * blocks).remainder(251).view(2, rows, blocks).to(torch.uint8)
    got = qmm.mx4_scales(plain)
    for i in range(2):
        assert np.array_equal(got[i].numpy(), ref.tiles(plain[i].numpy()))
    assert np.array_equal(qmm.mx4_scales(plain[0]).numpy(), got[0].numpy())


def test_scales_of_a_checkpoint_are_bytes():
    """A floating-point type's numbers are not its bits: 2 ** (byte - 127) would be made a whole number."""
    plain = torch.arange(100, 108, dtype=torch.uint8).view(2, 4)
    for bad in (plain.view(torch.float8_e8m0fnu), plain.float(), plain.bfloat16()):
        with pytest.raises(TypeError):
            qmm.mx4_scales(bad)
    bits = plain.view(torch.float8_e8m0fnu).view(torch.uint8)
    assert np.array_equal(qmm.mx4_scales(bits).numpy(), ref.tiles(plain.numpy()))


def test_reference_is_the_format():
    """The reference's own borders: halves go to the even code, 7 and more to 6, the sign of a zero stays."""
    x = np.zeros((1, 32))
    x[0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, -0.25, -0.75, -0.0, 0.2500001, 1.2500001, 5.1, 4.9]
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 127
    assert codes[0, :16].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 10, 8, 1, 3, 7, 6]
    assert ref.quantize(np.full((1, 32), 2.0 ** -126))[1][0, 0] == 0
    assert ref.quantize(np.full((1, 32), 2.0 ** 127))[1][0, 0] == 252
    assert ref.quantize(np.r_[np.inf, np.zeros(31)][None])[1][0, 0] == 255
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)


def test_timeout_hook_limits(L):
    for ns in (999, 100_000_001, -5):
        assert L.qmm_test_timeout_next_mx4(ns) == ARG


def test_cpu_tensors_are_refused(L):
    x, c, s = torch.zeros(4, 64), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(512, dtype=torch.uint8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: qmm.mx4_quantize(x), lambda: qmm.mx4_dequant(c, s), lambda: qmm.mx4_gemm(c, s, c, s),
                 lambda: qmm.moe_plan(x, 2), lambda: qmm.moe_quantize(x, i, 128), lambda: qmm.moe_combine(x, None, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        qmm.mx4_quantize(x.half())
