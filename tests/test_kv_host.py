"""Refusals of the key/value cache entry points, before any device memory is touched (no call here reaches a kernel)."""
import ctypes

import pytest

from quantized_weight_gb300 import build as qbuild
from quantized_weight_gb300 import qmm

OK, ARG, SHAPE, ALIGN, UNSUP = 0, -1, -2, -3, -4
FAKE, MIS, ODD = 0x10000, 0x10004, 0x10002


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qmm.lib()


def test_cache_size(L):
    assert L.qmm_kv_cache_size(3, 2, 128, 64, 64) == 3 * 2 * 4 * 2304
    assert L.qmm_kv_cache_size(1, 1, 64, 16, 32) == 16 * 64 + 128 * 2
    assert L.qmm_kv_cache_size(70000, 8, 256, 256, 32) == 70000 * 8 * 16 * (16 * 256 + 128 * 8)    # past 32 bits
    for bad in ((1, 1, 96, 16, 32), (1, 1, 128, 24, 64), (1, 1, 128, 8, 64), (1, 1, 128, 512, 64), (1, 1, 64, 16, 128),
                (1, 0, 64, 16, 64), (-1, 1, 64, 16, 64), (1 << 27, 1, 64, 16, 64)):
        assert L.qmm_kv_cache_size(*bad) == 0


def plan(L, cached=FAKE, fresh=FAKE, free=FAKE, n_free=4, table=FAKE, B=2, blocks=3, page=16, tokens=5, slots=FAKE,
         pos=FAKE, cu=FAKE, lens=FAKE, need=FAKE):
    return L.qmm_kv_plan(cached, fresh, free, n_free, table, B, blocks, page, tokens, slots, pos, cu, lens, need, None)


def test_plan_validation(L):
    for page in (0, 8, 48, 512, -16):
        assert plan(L, page=page) == UNSUP
    assert plan(L, B=-1) == SHAPE and plan(L, B=8193) == SHAPE
    assert plan(L, n_free=-1) == SHAPE and plan(L, blocks=-1) == SHAPE and plan(L, tokens=-1) == SHAPE
    for name in ("cached", "fresh", "free", "table", "slots", "pos", "cu", "lens", "need"):
        assert plan(L, **{name: None}) == ARG, name
        assert plan(L, **{name: ODD}) == ALIGN, name


def append(L, k=FAKE, v=FAKE, dt=0, kt=256, kh=128, vt=256, vh=128, slots=FAKE, cache=FAKE, T=4, pages=3, H=2, D=128,
           page=16, group=64):
    return L.qmm_kv_append(k, v, dt, kt, kh, vt, vh, slots, cache, T, pages, H, D, page, group, None)


def test_append_validation(L):
    assert append(L, dt=2) == UNSUP and append(L, D=96) == UNSUP and append(L, group=16) == UNSUP
    assert append(L, D=64, group=128) == UNSUP and append(L, page=20) == UNSUP
    assert append(L, T=-1) == SHAPE and append(L, pages=-1) == SHAPE and append(L, H=0) == SHAPE
    assert append(L, pages=1 << 27) == SHAPE
    for name in ("k", "v", "slots", "cache"):
        assert append(L, **{name: None}) == ARG, name
    for name in ("k", "v", "cache"):
        assert append(L, **{name: MIS}) == ALIGN, name
    assert append(L, slots=ODD) == ALIGN
    assert append(L, kt=258) == ALIGN and append(L, vh=130) == ALIGN
    assert append(L, dt=1, kt=260) == ALIGN                # 520 bytes: 8-byte steps only
    assert append(L, T=0) == OK and append(L, pages=0) == OK


def test_read_validation(L):
    def read(slots=FAKE, cache=FAKE, k=FAKE, v=FAKE, dt=0, T=4, pages=3, H=2, D=128, page=16, group=64):
        return L.qmm_kv_read(slots, cache, k, v, dt, T, pages, H, D, page, group, None)
    assert read(dt=-1) == UNSUP and read(D=32) == UNSUP and read(group=48) == UNSUP and read(page=15) == UNSUP
    assert read(T=-2) == SHAPE and read(H=-1) == SHAPE
    for name in ("slots", "cache", "k", "v"):
        assert read(**{name: None}) == ARG, name
    for name in ("cache", "k", "v"):
        assert read(**{name: MIS}) == ALIGN, name
    assert read(slots=ODD) == ALIGN
    assert read(T=0) == OK


def attend(L, q=FAKE, dt=0, qt=512, qh=128, cache=FAKE, table=FAKE, lens=FAKE, cu=FAKE, out=FAKE, T=5, B=2, blocks=3,
           most=4, pages=3, H=4, Hkv=2, D=128, page=16, group=64, scale=0.1, window=0, ws=FAKE, nbytes=1 << 30):
    return L.qmm_kv_attend(q, dt, qt, qh, cache, table, lens, cu, out, T, B, blocks, most, pages, H, Hkv, D, page, group,
                           scale, window, ws, nbytes, None)


def test_attend_validation(L):
    assert attend(L, dt=7) == UNSUP and attend(L, D=192) == UNSUP and attend(L, group=256) == UNSUP
    assert attend(L, page=0) == UNSUP
    assert attend(L, T=-1) == SHAPE and attend(L, B=-1) == SHAPE and attend(L, blocks=-1) == SHAPE
    assert attend(L, most=0) == SHAPE and attend(L, window=-1) == SHAPE
    assert attend(L, H=5) == SHAPE and attend(L, H=0) == SHAPE and attend(L, Hkv=0) == SHAPE
    assert attend(L, blocks=1 << 28) == SHAPE
    assert attend(L, cu=None) == SHAPE                     # without offsets every request has one query
    assert attend(L, cu=None, T=2, most=2) == SHAPE
    assert attend(L, scale=0.0) == ARG and attend(L, scale=-1.0) == ARG
    assert attend(L, scale=float("nan")) == ARG and attend(L, scale=float("inf")) == ARG
    for name in ("q", "cache", "table", "lens", "out", "ws"):
        assert attend(L, **{name: None}) == ARG, name
    for name in ("q", "cache", "out", "ws"):
        assert attend(L, **{name: MIS}) == ALIGN, name
    for name in ("table", "lens", "cu"):
        assert attend(L, **{name: ODD}) == ALIGN, name
    assert attend(L, qt=514) == ALIGN and attend(L, dt=1, qh=132) == ALIGN
    need = L.qmm_kv_attend_workspace_size(2, 4, 2, 128, 4)
    assert need >= 16 and attend(L, nbytes=need - 1) == SHAPE
    assert attend(L, T=0) == OK
    assert L.qmm_kv_attend_workspace_size(2, 5, 2, 128, 4) == 0
    assert L.qmm_kv_attend_workspace_size(2, 4, 2, 100, 4) == 0


def test_binding_refusals(L):
    import torch
    with pytest.raises(ValueError):
        qmm.kv_cache(3, 2, 100, 16)
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.kv_append(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(3, 2, 2304, dtype=torch.uint8), 16)
    with pytest.raises(TypeError):
        qmm.kv_append(x.half(), x.half(), torch.zeros(4, dtype=torch.int32), torch.zeros(3, 2, 2304, dtype=torch.uint8), 16)
