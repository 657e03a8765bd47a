"""Scales that leave fp32 once scores are taken in powers of two are refused on the host."""
import ctypes

import pytest

INVALID = 1
P = 1 << 20


@pytest.mark.parametrize("scale", [2.4e38, 3.0e38, 3.4e38])
def test_scales_beyond_fp32_in_powers_of_two(scale):
    """scale log2(e) is above fp32's largest number, 3.4028e38, from 2.3586e38 on."""
    from block_diffusion_speculative_hidden_gb300 import _lib, build_lib
    build_lib.build()
    kv = _lib.DflashPagedKV(P, P, P, P, 100, 5, 20, 2, 64, 1)
    assert _lib.lib().dflash_prefix_attention(ctypes.byref(kv), P, 256, 4, None, None, 3, 2, None, None, 0, 1, scale, 0,
                                              0, 2 * P, None, P, 1 << 40, None, None) == INVALID
