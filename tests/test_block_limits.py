"""Lengths at the end of 32-bit integers (host checks, no CUDA call): refused, not wrapped."""
import ctypes

import pytest

import sparse_mixed_precision_b200 as da2

MAX = 2 ** 31 - 1
LAST = MAX - 255                     # lengths are rounded up to 256 in 32 bits


def _size(fn, cfg):
    n = ctypes.c_size_t()
    return getattr(da2.lib(), fn)(ctypes.byref(cfg), ctypes.byref(n)), n.value


@pytest.mark.parametrize("Tq,Tk", [(MAX, 4096), (LAST + 1, 1), (4096, MAX), (1, LAST + 1), (MAX, MAX)])
def test_cross_attention_refuses_lengths_that_would_wrap(Tq, Tk):
    cfg = da2.cross_config(1, 1, Tq, Tk, 64)
    for fn in ("da2_cross_attention_workspace_size", "da2_cross_attention_backward_workspace_size"):
        assert _size(fn, cfg) == (2, 0)


def test_cross_attention_workspace_of_the_longest_lengths():
    assert _size("da2_cross_attention_workspace_size", da2.cross_config(1, 1, LAST, 4096, 64)) == (0, 256)
    status, n = _size("da2_cross_attention_backward_workspace_size", da2.cross_config(1, 1, LAST, 4096, 64))
    assert status == 0 and n >= 2 * 4 * LAST            # lse and D of every row
    status, n = _size("da2_cross_attention_workspace_size", da2.cross_config(1, 1, 1, LAST, 64))
    assert status == 0 and 256 < n < 1 << 20            # split over the keys


def test_norm_refuses_lengths_that_would_wrap():
    assert _size("da2_qk_norm_rope_workspace_size", da2.norm_rope_config(1, 1, 0, MAX, 64, T_rot=0))[0] == 2
    assert _size("da2_qk_norm_rope_workspace_size", da2.norm_rope_config(1, 1, 0, LAST + 1, 64, T_rot=0))[0] == 2
    assert _size("da2_qk_norm_rope_workspace_size", da2.norm_rope_config(1, 1, 0, LAST, 64, T_rot=0))[0] == 0
