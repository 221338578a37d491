"""Host checks of sd_cache_attn's scale: scores are formed in powers of two, so
scale * log2(e) has to be finite too.  Nothing reaches the GPU."""

import ctypes

import pytest

import draft_verification_amd as sdv
from draft_verification_amd import _lib


@pytest.mark.parametrize("scale,code", [(3.4e38, _lib.SD_EINVAL), (2.4e38, _lib.SD_EINVAL), (2.3e38, _lib.SD_OK),
                                        (1e-45, _lib.SD_OK), (1.0, _lib.SD_OK), (0.0, _lib.SD_EINVAL)])
def test_scales(scale, code):
    at = [ctypes.c_void_p((i + 1) << 44) for i in range(10)]
    got = sdv.lib().sd_cache_attn(None, 3, 2, 4, 2, 64, 0, at[0], 256, _lib.SD_CACHE_BF16, 16, 8, at[1], at[2], at[3], at[4],
                                  at[5], 4, scale, at[6], 256, at[7], at[8], at[9], 1 << 30)   # no rows
    assert got == code
