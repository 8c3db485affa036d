"""Both sides of the cache calls' limits, as include/qmm.h states them.  A size on the right side is shown by the refusal that
comes after it (a missing pointer), so that no call here reaches a kernel."""
import pytest

from quantized_weight_gb300 import qmm
from test_kv_host import ARG, L, SHAPE, append, attend, plan  # noqa: F401


def test_tokens(L):
    for T, want in (((1 << 19) - 1, ARG), (1 << 19, SHAPE)):
        assert append(L, T=T, k=None) == want
        assert L.qmm_kv_read(None, 0x10000, 0x10000, 0x10000, 0, T, 3, 2, 128, 16, 64, None) == want
        assert attend(L, T=T, q=None) == want
        assert attend(L, most=T, q=None) == want
    for T, want in (((1 << 31) - 1, ARG), (1 << 31, SHAPE)):
        assert plan(L, tokens=T, slots=None) == want


def test_heads(L):
    assert append(L, H=4096, k=None) == ARG and append(L, H=4097, k=None) == SHAPE
    assert attend(L, H=1024, q=None) == ARG and attend(L, H=1026, q=None) == SHAPE
    assert L.qmm_kv_cache_size(1, 4096, 64, 16, 64) > 0 and L.qmm_kv_cache_size(1, 4097, 64, 16, 64) == 0


@pytest.mark.parametrize("page", [16, 64, 256])
def test_positions(L, page):
    last = (1 << 31) // page
    assert append(L, pages=last - 1, page=page, k=None) == ARG and append(L, pages=last, page=page, k=None) == SHAPE
    fits = ((1 << 31) - 256) // page
    assert attend(L, blocks=fits, page=page, q=None) == ARG and attend(L, blocks=fits + 1, page=page, q=None) == SHAPE
    assert attend(L, blocks=1 << 62, page=page, q=None) == SHAPE      # past 64 bits as a number of positions


def test_plan_limits(L):
    assert plan(L, B=8192, cached=None) == ARG and plan(L, B=8193, cached=None) == SHAPE
    assert plan(L, n_free=(1 << 31) - 1, free=None) == ARG and plan(L, n_free=1 << 31, free=None) == SHAPE
    assert plan(L, blocks=(1 << 31) - 1, table=None) == ARG and plan(L, blocks=1 << 31, table=None) == SHAPE


def test_workspace_has_a_size_where_attend_has_a_call(L):
    size = L.qmm_kv_attend_workspace_size
    assert size(2, 1024, 1, 128, 1) > 0 and size(2, 1025, 1, 128, 1) == 0
    assert size(2, 4, 2, 128, (1 << 19) - 1) > 0 and size(2, 4, 2, 128, 1 << 19) == 0
    assert size((1 << 31) - 1, 4, 2, 128, 1) > 0 and size(1 << 31, 4, 2, 128, 1) == 0
    with pytest.raises(ValueError):
        qmm.kv_attend_workspace(1, 2048, 1, 128, device="cpu")


def test_empty_cache_has_a_page_size(L):
    assert qmm.kv_cache(0, 2, 128, 64, device="cpu").shape == (0, 2, qmm.kv_cache(3, 2, 128, 64, device="cpu").shape[2])
    for bad in ((0, 2, 100, 64), (0, 0, 128, 64), (-1, 2, 128, 64), (0, 2, 128, 24)):
        with pytest.raises(ValueError):
            qmm.kv_cache(*bad, device="cpu")


def test_timeout_hook_limits(L):
    for ns in (999, 100_000_001, -5):
        assert L.qmm_test_timeout_next_attend(ns) == ARG
