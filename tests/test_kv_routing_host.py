"""Which kernel takes an attention call: the rule's borders, and the kernel that the GPU tests mean.  Without a device the rule
counts a GB300's 152 SMs."""
import pytest
import torch

from quantized_weight_gb300 import qmm
from test_kv_host import L, SHAPE, UNSUP  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32


def tiles(B, H, Hkv, D, most, dtype=BF16):
    return qmm.kv_attend_tiles(dtype, B, H, Hkv, D, most)


@pytest.mark.parametrize("D,small,large", [(64, 4500, 8000), (128, 3900, 6200), (256, 3200, 3200)])
def test_borders(L, D, small, large):
    # items of one kv head with up to 128 rows, in one round of the SMs and in two
    for rows, border in ((100, small), (128, small), (129, large), (250, large)):
        per = 128 if D == 256 else 256
        a = -(-rows // per)                                # items a request
        B = border // rows
        assert B * a <= 152
        assert not tiles(B, rows, 1, D, 1) and tiles(B + 1, rows, 1, D, 1)
        B = 152 // a
        assert tiles(B, rows, 1, D, 1)                     # the last of one round; the next one counts for two
        assert tiles(B + 1, rows, 1, D, 1) == ((B + 1) * rows > 2 * border)


def test_few_rows_and_float32_stay(L):
    for D in (64, 128, 256):
        assert not tiles(8000, 16, 1, D, 1) and not tiles(4000, 32, 4, D, 2)
        assert not tiles(1, 32, 8, D, 4096, F32) and tiles(1, 32, 8, D, 4096)


def test_refusals(L):
    f = L.qmm_kv_attend_tiles
    assert f(2, 1, 4, 2, 128, 1) == UNSUP and f(1, 1, 4, 2, 96, 1) == UNSUP
    for bad in ((1, -1, 4, 2, 128, 1), (1, 1, 5, 2, 128, 1), (1, 1, 0, 2, 128, 1), (1, 1, 2048, 2, 128, 1), (1, 1, 4, 2, 128, 0),
                (1, 1, 4, 2, 128, 1 << 19)):
        assert f(*bad) == SHAPE
    with pytest.raises(qmm.QmmError):
        tiles(1, 5, 2, 128, 1)
    with pytest.raises(TypeError):
        tiles(1, 4, 2, 128, 1, torch.float16)


def test_the_gpu_tests_of_the_prompt_kernel_reach_it(L):
    """Sizes (B, H, Hkv, most) of the tests that are there for it."""
    for D in (64, 128, 256):
        for case in ((5, 16, 2, 130), (2, 33, 1, 140),     # test_attend_many_rows
                     (30, 40, 5, 8),                       # ..._of_few_tokens
                     (2, 64, 2, 130),                      # ..._small_large_and_missing
                     (1, 64, 2, 140),                      # test_attend_non_finite_values and the edges
                     (1, 72, 2, 128),                      # test_many_small_probabilities_beside_a_large_one
                     (80, 32, 8, 64), (70, 32, 8, 150),    # items one after the other
                     (80, 32, 8, 20)):                     # test_wait_runs_out_then_the_next_call_is_normal
            assert tiles(*case[:3], D, case[3]), (D, case)
    assert tiles(1, 32, 8, 128, 1300)                      # test_large_cache
