"""The decode-step calls at the ends of what they accept and in every variant of
their kernels, against 64-bit definitions.  Tolerances are those derived in
tests/test_gpu_decode_step.py, where nothing else is said."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import LOST, U, attend_inputs, dev, dtype_of, host, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- attention -------------------------------------------------------------------

def test_attention_of_more_items_than_a_grid_axis_holds(tb):  # noqa: F811
    """2^24 and more (row, key/value head) pairs, with 256 threads each, are 2^32
    threads, which one axis of a grid does not hold.  Every output is looked at."""
    import torch
    T, kv, D, ps, scale = (1 << 22) + 77, 4, 64, 8, 0.2
    base = [23, 1, 0, 17]
    say(f"[range] attention of {T} rows, {kv} heads")
    caches, tables, _, ks, vs = attend_inputs(2, base, 4, kv, 1, D, ps, "bf16")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(1)
    q = torch.randn(T, kv * D, generator=gen, device="cuda:0")
    rows = torch.randint(-1, 5, (T,), generator=gen, device="cuda:0", dtype=torch.int32)
    most = torch.tensor(base + [0], device="cuda:0")[torch.where((rows < 0) | (rows > 3), 4, rows)]
    lens = (torch.rand(T, generator=gen, device="cuda:0") * (most + 1)).int()
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, q, dev(tables), lens, scale=scale,
                                         rows=rows, return_lse=True)
    torch.cuda.synchronize()
    say("[range] launched")
    for t0 in range(0, T, 1 << 20):
        part = slice(t0, min(T, t0 + (1 << 20)))
        r, n = rows[part], lens[part].double()
        for h in range(kv):
            x = q[part, h * D:(h + 1) * D].double()
            want = torch.zeros_like(x)
            tol = torch.zeros_like(x)
            e = torch.full_like(n, -float("inf"))
            big = torch.zeros_like(n)
            for row in range(4):
                k, v = dev(ks[row][h]), dev(vs[row][h])
                there = (torch.arange(base[row], device="cuda:0") < n[:, None]) & (r == row)[:, None]
                if base[row] == 0:
                    continue
                s = (scale * (x @ k.T.contiguous())).masked_fill(~there, -float("inf"))
                here = there[:, 0]
                size = (scale * (x.abs() @ k.abs().T.contiguous())).masked_fill(~there, 0).amax(1)
                p = torch.softmax(s, 1)
                want = torch.where(here[:, None], p @ v, want)
                factor = U * (2 * (D + 16) * size + 2 * n + 64)
                tol = torch.where(here[:, None], factor[:, None] * (p @ v.abs()), tol)
                e = torch.where(here, torch.logsumexp(s, 1), e)
                big = torch.where(here, size, big)
            assert ((out[part, h * D:(h + 1) * D] - want).abs() <= tol).all().item(), (t0, h)
            got, none = lse[part, h].double(), e == -float("inf")
            bound = U * ((D + 16) * big + n + 64 + 2 * e.abs())
            assert torch.equal(got == -float("inf"), none)
            assert ((got - e).abs() <= bound)[~none].all().item(), (t0, h)
