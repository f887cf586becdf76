"""Rows whose maximum moves across 2^20, where the sums' exponents change their form,
between the tiles of a workgroup, its waves and the chunks of a row."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import check_select, say, tb  # noqa: F401
from tests.test_gpu_prompt import check_logprobs

pytestmark = pytest.mark.gpu


def rows(R, V):
    ramp = np.linspace(-60, 60, V)
    one = np.stack([2.0 ** 20 + ramp, 2.0 ** 20 - ramp, -2.0 ** 20 + ramp, -2.0 ** 20 - ramp,
                    np.where(ramp < 0, 5 + ramp, 2.0 ** 21), np.where(ramp < 0, -1e30, ramp),
                    np.where(ramp < 0, -np.inf, 1e7 + ramp)])
    return np.tile(one, (-(-R // len(one)), 1))[:R].astype(np.float32)


@pytest.mark.parametrize("R,V", [(7, 40000), (7, 5000), (1029, 12289)])
def test_logprobs_across(tb, R, V):  # noqa: F811
    say(f"[logprobs] maxima across 2^20, {R} x {V}")
    x = rows(R, V)
    check_logprobs(tb, x, np.full(R, V - 1, np.int32), 3)


@pytest.mark.parametrize("R,V", [(7, 40000), (7, 5000), (1029, 12289)])
def test_select_across(tb, R, V):  # noqa: F811
    say(f"[select] maxima across 2^20, {R} x {V}")
    check_select(tb, rows(R, V), np.full(R, -3.0, np.float32), 1, exact_ties=True)
