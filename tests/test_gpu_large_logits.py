"""Beam selection over logits far from zero: masks of -1e30 that fill a row, and
logits whose size leaves one fp32 step of a unit or more."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import check_select, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [7, 5000, 40000])
@pytest.mark.parametrize("rows", [1, 30])
def test_select_far_from_zero(tb, V, rows):  # noqa: F811
    say(f"[select] far from zero, {rows} times, V={V}")
    ramp = np.linspace(-60, 60, V)
    x = np.stack([np.full(V, -1e30), np.full(V, 1e30), 2.0 ** 24 + ramp, 2.0 ** 20 + ramp,
                  -2.0 ** 20 - ramp, np.full(V, np.finfo(np.float32).min), 1e10 + 1e4 * ramp,
                  np.full(V, 3e9)] * rows).astype(np.float32)
    x[1, :-1] = -1e30
    scores = np.full(len(x), -3.0, np.float32)
    check_select(tb, x, scores, 1, exact_ties=True)
