"""Scales that the attention calls take and refuse: scores are computed in units of log 2."""
import ctypes
import math

import pytest

from tests.test_decode_step_host import A, GB, L, cache  # noqa: F401
from tests.test_prompt_host import PASSED, SHAPE, chunk


def attend(L, scale):  # noqa: F811
    ws = L.bitnet_paged_attention_workspace_bytes(4, 12, 2, 128, 512)
    return L.bitnet_paged_attention(ctypes.byref(cache(k=A + 6 * GB, v=A + 7 * GB)), 0, 4, 12, A, 1536,
                                    A + GB, 4, 8, None, A + 2 * GB, 512, scale, A + 3 * GB, None,
                                    A + 4 * GB, ws, None)


@pytest.mark.parametrize("call", [attend, lambda L, s: chunk(L, sc=s)])
def test_scales(L, call):  # noqa: F811
    largest = 2.0 ** 128 / math.log2(math.e)
    for ok in (0.0, -0.0, 0.1, -3.0, 1e-45, -1e-40, 2.0 ** 127, -2.0 ** 127, 0.999999 * largest):
        assert call(L, ok) in PASSED, ok
    for bad in (1.000001 * largest, -1.000001 * largest, 3.4e38, math.inf, -math.inf, math.nan):
        assert call(L, bad) == SHAPE, bad
