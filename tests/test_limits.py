"""Sizes at the edge of what the kernels count in 32 bits (no GPU needed)."""
import ctypes

import pytest
import torch

MOST = 2 ** 31 - 1 - 8192   # tokens of one sequence that fa_mask_ranges takes


def _ranges(fa, S):
    vp = ctypes.c_void_p
    return fa.lib().fa_mask_ranges(vp(0x2000), None, 0, 1, S, 1, -1, -1, vp(0x100000), 1 << 60, None)


@pytest.mark.parametrize("S", [MOST + 1, 2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 1])
def test_mask_ranges_too_long(fa, S):
    """Rows rounded up, or a search step past the last one, would leave 32 bits: no
    size, and no call with such a buffer."""
    assert fa.lib().fa_mask_ranges_bytes(1, S) == 0
    assert _ranges(fa, S) == fa.FA_ERR_INVALID_ARG
    e = fa.FaExt(window_left=-1, window_right=-1)
    e.mask_ranges, e.mask_ranges_bytes = 0x100000, 1 << 60
    p = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(5)]
    assert fa.lib().fa_fwd_ext(*p, 1, S, S, 1, 1, 64, 0.125, 0, None, None, ctypes.byref(e), 0, None) == \
        fa.FA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the longest call is looked at on a machine without a GPU")
def test_mask_ranges_longest(fa):
    n = fa.lib().fa_mask_ranges_bytes(1, MOST)
    rows = (MOST + 127) // 128 * 128
    assert n > rows * 8 and rows < 2 ** 31
    assert _ranges(fa, MOST) != fa.FA_ERR_INVALID_ARG   # (no device here)
