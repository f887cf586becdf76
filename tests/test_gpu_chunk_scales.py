"""Chunk attention where the scale and the queries lie far apart: their product is what
counts, and it is near one, tiny or zero."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import say, tb  # noqa: F401
from tests.test_gpu_prompt import Paged, run_chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("q2,s2", [(-120, 15), (-120, 118), (-149, 125), (-100, 97), (-60, 57),
                                   (120, -123), (-113, 14), (-115, 13)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_of_far_scales(tb, dtype, q2, s2, D):  # noqa: F811
    """Some heads are zeros: they give the mean of the values."""
    say(f"[chunk] {dtype} {D} queries 2^{q2}, scale 2^{s2}")
    rng = np.random.default_rng(D + abs(q2))
    new, old = np.array([40, 1, 9]), np.array([3, 70, 300])
    pg = Paged(tb, rng, dtype, new + old, 2, D, 16)
    q = np.ldexp(rng.normal(0, 1, (50, 6, D)), q2).astype(np.float32)
    q[:, 1], q[7] = 0, 0
    out, _ = run_chunk(tb, pg, q, np.r_[0, np.cumsum(new)], new + old, 6, scale=2.0 ** s2)
    assert np.isfinite(out).all()
