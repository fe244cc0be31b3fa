"""The attention's softmax scale at the ends of fp32, without a GPU: the kernels multiply it by
log2(e), so what would overflow there is refused like an infinite one."""
import ctypes

import numpy as np
import pytest

from mxfp_block_scaled_b200 import mxq

P = 0x1000                  # never dereferenced: every call below fails a check before any launch
LARGEST = float(np.finfo(np.float32).max)


def call(scale):
    cache = mxq._CacheStruct(P, P, P, P, None, None, 4, 2, 16, 64, mxq.FMT["mxfp8"])
    return mxq.load().mxq_cache_attention(ctypes.byref(cache), P, 256, 2, 4, P, P, P, 1, 1, 2, scale, P, P, P, None, 0, None)


@pytest.mark.parametrize("scale", [LARGEST, -LARGEST, float(np.nextafter(np.float32(2.0 ** 127), np.float32(np.inf))), float("inf"), float("nan")])
def test_scales_that_leave_fp32_are_refused(scale):
    assert call(scale) == 1


@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127, 0.0, 1e-45])
def test_scales_within_it_go_on_to_the_next_check(scale):
    assert np.isfinite(np.float32(scale) * np.float32(1.4426950408889634))
    assert call(scale) == 4         # no workspace
