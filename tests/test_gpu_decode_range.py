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


def stretches(lens, kv, G, D, max_len):
    """How the kernel cuts the tiles of these rows: "items" (a workgroup each),
    "apart" (every item starts a stretch) or "shared" (stretches hold parts of
    several items), and the tiles of a stretch.  The rule that the kernel's comments
    give, for choosing inputs that reach each case."""
    T, row_items = len(lens), kv * (-(-G // 16))
    items, tiles = T * row_items, -(-max_len // 32)
    if T > 1024 or items * tiles >= 1 << 30:
        return "items", 0
    grid = min(2048 if 2 * items > 512 else 256 if D == 256 else 512, items * (tiles // 4 + 2))
    per = [-(-int(n) // 32) for n in lens]
    raw, most = sum(per) * row_items, max(per)
    rounds = lambda n: -(-n // 4) * 4
    least = most // 254 + 1
    stretch = rounds(max(-(-raw // 256), 12 if most <= 12 else 1, least))
    if stretch <= 16 and items * stretch + raw <= grid * stretch:
        return "apart", stretch
    return "shared", rounds(max(-(-raw // grid), 8, least))


def check_rows(out, lse, q, rows, lens, ks, vs, scale, D, lost):
    """Every output against 64-bit arithmetic, a key/value head's queries at once."""
    T, kv = len(rows), ks[0].shape[0]
    H = q.shape[1] // D
    out, q = out.reshape(T, kv, -1, D), q.reshape(T, kv, -1, D).astype(np.float64)
    lse = lse.reshape(T, kv, -1)
    kabs, vabs = [np.abs(k) for k in ks], [np.abs(v) for v in vs]
    for t in range(T):
        n = int(lens[t])
        if n == 0:
            assert (out[t] == 0).all() and (lse[t] == -np.inf).all(), t
            continue
        for h in range(kv):
            k, v = ks[rows[t]][h, :n], vs[rows[t]][h, :n]
            s = scale * (q[t, h] @ k.T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            e = (m + np.log(total))[:, 0]
            p /= total
            size = (scale * (np.abs(q[t, h]) @ kabs[rows[t]][h, :n].T)).max(1)
            tol = U * (2 * (D + 16) * size + 2 * n + 64)[:, None] * (p @ vabs[rows[t]][h, :n])
            tol += n * lost * vabs[rows[t]][h, :n].max()
            err = np.abs(out[t, h] - p @ v)
            assert (err <= tol).all(), (t, h, n, float((err / tol).max()))
            bound = U * ((D + 16) * size + n + 64 + 2 * np.abs(e))
            assert (np.abs(lse[t, h] - e) <= bound).all(), (t, h, n)
    assert H == kv * out.shape[2]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [5, 17])
@pytest.mark.parametrize("cut,T", [("shared", 40), ("shared", 150), ("apart", 70), ("items", 1030)])
def test_attention_in_every_variant(tb, dt, D, G, cut, T):  # noqa: F811
    """Each type, head size and product layout with up to 64 rows, with more and with
    more than 1024, in stretches that items share, that they begin and alone."""
    import torch
    say(f"[range] attention {dt} D={D} G={G} T={T} {cut}")
    kv, ps = 2, 32
    base = {40: [3500, 2900, 1200, 33], 150: [1300, 900, 65, 7], 70: [300, 150, 64, 1],
            1030: [70, 40, 33, 1]}[T]
    caches, tables, _, ks, vs = attend_inputs(T + D, base, -(-base[0] // ps) + 1, kv, G, D, ps, dt,
                                              hf=D != 128)
    rng = np.random.default_rng(T + G)
    rows = rng.choice(4, T, p=[0.5, 0.3, 0.1, 0.1]).astype(np.int32)
    lens = np.array([rng.integers(base[r] // 2 + 1, base[r] + 1) for r in rows], np.int32)
    lens[rng.permutation(T)[:T // 12]] = 0
    got, stretch = stretches(lens, kv, G, D, tables.shape[1] * ps)
    assert got == cut
    if cut == "shared":   # of which many hold the end of one item and the start of another
        ends = np.cumsum(np.repeat(-(-lens // 32), kv * (-(-G // 16))))
        assert ((ends % stretch) != 0).sum() > len(lens)
    q = rng.normal(0, 1, (T, kv * G * D)).astype(np.float32)
    cache = tb.KvCache(*caches)
    first = None
    for _ in range(2):
        out, lse = tb.bitnet_paged_attention(cache, 1, dev(q), dev(tables), dev(lens),
                                             rows=dev(rows), return_lse=True)
        assert first is None or torch.equal(first, out)
        first = out
    check_rows(host(out), host(lse), q, rows, lens, ks, vs, D ** -0.5, D, LOST[dt])
