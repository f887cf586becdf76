"""Chunk attention at the ends of what the header allows: large 8-bit values at lengths
whose sums would pass fp32's range, large 8-bit keys, large bf16 values.

All tokens have the same values, so that every row's output is that of one token, and
keys alternate from page to page between a score of 0 and one of 4.1, which is less than
2^6 times as likely, so that a base that the first page has set stays: with u = 2^-24 the
sums of n tokens are off by n u relative each and the output by twice that, apart from 64
u for the terms and the joins; lse by n u and 64 u, S = 4.1 as tests/test_gpu_prompt.py
has it."""
import math

import numpy as np
import pytest

from tests.test_gpu_decode_step import U, dev, host, say, tb  # noqa: F401
from tests.test_gpu_prompt import Paged, run_chunk

pytestmark = pytest.mark.gpu
PS, HIGH = 64, 4.1


def alternating(tb, dtype, D, R, new, n, value):  # noqa: F811
    """R requests of n tokens, `new` of them new, on the same two pages."""
    import torch
    rng = np.random.default_rng(D + R)
    f = lambda *s: torch.empty(*s, device="cuda:0")
    i32 = lambda a: dev(np.asarray(a).astype(np.int32))
    if dtype == "int8":
        code = rng.integers(-127, 128, D)
        code[:2] = 127, -127
        k, v = (torch.zeros(1, 2, 1, PS, D, dtype=torch.int8, device="cuda:0") for _ in range(2))
        k[0, 1] = 1
        v[:] = dev(code.astype(np.int8))
        cache = tb.KvCache(k, v, f(1, 2, 1, PS).fill_(HIGH / D), f(1, 2, 1, PS).fill_(value / 127))
        row, key = code * float(np.float32(value / 127)), float(np.float32(HIGH / D))
    else:
        sign = rng.choice([-1.0, 1.0], D)
        k, v = (torch.zeros(1, 2, 1, PS, D, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
        k[0, 1] = HIGH / D
        v[:] = dev((sign * value).astype(np.float32)).bfloat16()
        cache, row, key = tb.KvCache(k, v), v[0, 0, 0, 0].double().cpu().numpy(), float(k[0, 1, 0, 0, 0])
    mp = -(-n // PS)
    tables = np.tile(np.arange(mp) % 2, (R, 1))
    T = R * new
    q = torch.ones(T, D, device="cuda:0")
    out, lse = tb.bitnet_chunk_attention(cache, 0, q, i32(new * np.arange(R + 1)), i32(np.full(R, n)),
                                         i32(tables), n, 1.0, return_lse=True)
    sees = np.tile(n - new + 1 + np.arange(new), R)
    high = sees // (2 * PS) * PS + np.maximum(sees % (2 * PS) - PS, 0)
    want = np.log(high * math.exp(key * D) + sees - high)
    assert np.isfinite(host(out)).all()
    assert (np.abs(host(out) - row) <= U * (2 * n + 64) * np.abs(row)).all()
    assert (np.abs(host(lse)[:, 0] - want) <= U * ((D + 16) * HIGH + n + 64 + want)).all()


# Behind 17,400 tokens the sums pass 2^128; one token's length is cut, of 600 some are not.
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,new", [(1, 1), (1, 200), (600, 1), (70, 3)])
def test_large_values_of_8_bits(tb, D, R, new):  # noqa: F811
    say(f"[chunk] values of 2^100, {D} channels, {R} requests of {new}")
    alternating(tb, "int8", D, R, new, 32001, 0.999 * 2.0 ** 100)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,new", [(1, 1), (300, 2)])
def test_large_values_of_bf16(tb, D, R, new):  # noqa: F811
    say(f"[chunk] bf16 values of 2^112, {D} channels, {R} requests of {new}")
    alternating(tb, "bf16", D, R, new, 510, 2.0 ** 112)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_keys_of_8_bits(tb, D):  # noqa: F811
    """Keys just below 2^100 beside queries that make their scores ordinary."""
    say(f"[chunk] keys of 2^100, {D} channels")
    rng = np.random.default_rng(D)
    new, old = np.array([70, 1, 40]), np.array([0, 90, 300])
    pg = Paged(tb, rng, "int8", new + old, 2, D, 16)
    pg.ksd *= 2.0 ** 97
    pg.ks = host(pg.ksd)
    pg.make(tb)
    assert 2.0 ** 99 < np.abs(pg.k).max() < 2.0 ** 100
    q = (rng.normal(0, 1, (111, 6, D)) * 2.0 ** -97).astype(np.float32)
    run_chunk(tb, pg, q, np.r_[0, np.cumsum(new)], new + old, 6)
