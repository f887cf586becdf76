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
            size = (abs(scale) * (np.abs(q[t, h]) @ kabs[rows[t]][h, :n].T)).max(1)
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


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("T,kv,G,longest", [(3, 96, 1, 600), (2, 256, 2, 60), (70, 70, 2, 90),
                                            (5, 70, 20, 130), (66, 40, 33, 200)])
def test_attention_of_many_items_a_row(tb, dt, T, kv, G, longest):  # noqa: F811
    """More than 64 key/value heads (times groups of 16 query heads) a row."""
    D, ps = 64, 16
    say(f"[range] attention {dt} T={T} kv={kv} G={G}")
    base = [longest, longest // 2 + 1, 33]
    caches, tables, _, ks, vs = attend_inputs(kv, base, -(-longest // ps), kv, G, D, ps, dt)
    rng = np.random.default_rng(T)
    rows = rng.integers(0, 3, T).astype(np.int32)
    lens = np.array([rng.integers(1, base[r] + 1) for r in rows], np.int32)
    lens[T // 2] = 0
    q = rng.normal(0, 1, (T, kv * G * D)).astype(np.float32)
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables), dev(lens),
                                         rows=dev(rows), return_lse=True)
    check_rows(host(out), host(lse), q, rows, lens, ks, vs, D ** -0.5, D, LOST[dt])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.25, 1e-30, -3.0])
def test_attention_of_any_scale(tb, dt, scale):  # noqa: F811
    say(f"[range] attention {dt} scale {scale}")
    kv, G, D, ps = 2, 3, 128, 16
    caches, tables, q, ks, vs = attend_inputs(4, [300, 65, 1], 20, kv, G, D, ps, dt)
    lens = np.array([300, 65, 1], np.int32)
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables), dev(lens),
                                         scale=scale, return_lse=True)
    check_rows(host(out), host(lse), q, np.arange(3), lens, ks, vs, scale, D, LOST[dt])


@pytest.mark.parametrize("q2,k2,v2", [(-100, 100, 0), (118, -118, 0), (100, -100, -110), (0, 0, 120),
                                      (58, 58, 0), (50, 50, 100)])
def test_attention_of_any_magnitude(tb, q2, k2, v2):  # noqa: F811
    """bf16 caches near the ends of fp32: queries 2^-100 to 2^118, scores up to 2^122."""
    import torch
    say(f"[range] attention of q 2^{q2}, k 2^{k2}, v 2^{v2}")
    kv, G, D, ps, lens = 2, 3, 64, 16, np.array([70, 33, 600], np.int32)
    caches, tables, q, ks, vs = attend_inputs(6, lens.tolist(), 40, kv, G, D, ps, "bf16")
    for c, f, vals in ((caches[0], k2, ks), (caches[1], v2, vs)):
        c.copy_(torch.ldexp(c.float(), torch.tensor(f, device="cuda:0")).bfloat16())
        for x in vals:
            x *= 2.0 ** f
    q *= np.float32(2.0 ** q2)
    scale = 0.125
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables), dev(lens),
                                         scale=scale, return_lse=True)
    check_rows(host(out), host(lse), q, np.arange(3), lens, ks, vs, scale, D, LOST["bf16"])


# ---- beam selection: streams of many tiles ---------------------------------------

TILE = 4096


def tiles_of(rows, V):
    """Tiles that a workgroup takes one after the other, by the rule at the kernel's
    plan."""
    every = -(-V // TILE)
    return -(-every // min(every, 64, -(-1024 // rows)))


def select_exactly(x, scores, W, finished, eos):
    """The definition for large vocabularies, fp64; and the smallest gap between
    scores of different beams, up to the first that is left out."""
    R, V = x.shape
    out = {"scores": np.empty(R), "tokens": np.empty(R, np.int32), "parents": np.empty(R, np.int32),
           "finished": np.empty(R, np.int32)}
    gap = np.inf
    for g in range(0, R, W):
        cand = []
        for r in range(g, g + W):
            base = float(scores[r])
            if finished[r]:
                cand.append((-base, r, 0.0, eos))
                cand += [(np.inf, r, 0.0, t) for t in range(W + 1) if t != eos]
                continue
            y = np.where(x[r] < np.inf, x[r], -np.inf)
            m = np.float64(y.max())
            lse = m + np.log(np.exp(y.astype(np.float64) - m).sum()) if m > -np.inf else 0.0
            at = np.flatnonzero(y >= np.partition(y, V - W)[V - W])
            at = at[np.argsort(-y[at], kind="stable")][:W]
            cand += [(-(base + (np.float64(y[t]) - lse)), r, -y[t], int(t)) for t in at]
        cand.sort()
        for a, b in zip(cand[:W], cand[1:W + 1]):
            if a[1] != b[1] and a[0] < np.inf and a[0] != b[0]:
                gap = min(gap, b[0] - a[0])
        for j, (s, r, _, t) in enumerate(cand[:W]):
            out["scores"][g + j], out["tokens"][g + j], out["parents"][g + j] = -s, t, r
            out["finished"][g + j] = int(bool(finished[r]) or t == eos)
    return out, gap


# What a row's logits look like, by token.  "stairs": every tile is above all before
# it, so that each replaces what the lists hold and raises the maximum; "rising": so
# do a tile's threads, a few at a time, until the lists are cut; "clumps": so do all
# the logits of a few threads, and the lists are cut again and again; "holes": whole
# tiles, the first among them, with no token that can be taken, or NaN; "dust": one
# logit a thread and behind it terms that fp32 sums lose.
def pattern(kind, rng, R, W, V):
    i = np.arange(V)
    if kind == "random":
        x = rng.normal(0, 2, (R, V))
    elif kind == "rising":
        x = i * (30.0 / V) + rng.uniform(0, 8, (R, 1))
    elif kind == "falling":
        x = -i * (30.0 / V) + rng.uniform(0, 8, (R, 1))
    elif kind == "stairs":
        x = i // TILE * 1.5 + rng.random((R, V))
    elif kind == "clumps":   # (a thread's logits are four by four, 1024 apart)
        few = rng.random((R, -(-V // TILE), 256)) < (0.75 * min(max(W, 8), 32) / 64)
        x = np.where(few[:, i // TILE, i % 1024 // 4], i // TILE * 1.5, -3.0) + rng.random((R, V))
    elif kind == "equal":
        x = np.repeat(rng.normal(0, 2, (R, 1)), V, 1)
    elif kind == "holes":
        x = rng.normal(0, 2, (R, V))
        for r in range(R):
            gone = rng.random(-(-V // TILE)) < 0.5
            gone[0] = True
            x[r, np.repeat(gone, TILE)[:V]] = (-np.inf, np.nan, np.inf)[r % 3]
    else:
        x = np.where(i < 1024, 0.0, -18.1) + rng.uniform(0, 1e-3, (R, V))
    return np.ascontiguousarray(x, np.float32)


SHAPES = [(32, 8, 151936), (8, 8, 151936), (256, 4, 20000), (70, 3, 65537), (700, 1, 30001),
          (32, 32, 40000), (12, 12, 151936), (22, 12, 70000)]
KINDS = ["random", "rising", "falling", "stairs", "clumps", "equal", "holes", "dust"]


def stream_inputs(shape, kind):
    B, W, V = shape
    rng = np.random.default_rng(B * 37 + W + KINDS.index(kind))
    x = pattern(kind, rng, B * W, W, V)
    scores = (-3 - 9 * rng.random(B * W)).astype(np.float32)
    finished = (rng.random(B * W) < 0.1).astype(np.int32) * 3
    return x, scores, finished, int(rng.integers(0, V))


def sum_error(rows, V):
    """Relative error of a row's sum of exp in fp32, in units of u = 2^-24, and so the
    absolute error of its logarithm.  The arguments' roundings, u times the distance
    to the largest logit, weigh up to ln V on average; the constant log2 e is off
    by less than u, which again counts up to ln V; an exponential 2 u, one for the
    term and one for each of a thread's n - 1 and the two joins' rescalings; 4
    for the sum of 16, two for each further tile (a product and a sum), one
    for the rescaling to the chunk's maximum, 8 for the sums over lanes and
    waves."""
    n = tiles_of(rows, V)
    return 2 * np.log(V) + 2 * (n + 2) + 4 + 2 * (n - 1) + 1 + 8


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_select_streams_of_many_tiles(tb, shape, kind):  # noqa: F811
    import torch
    B, W, V = shape
    say(f"[range] selection B={B} W={W} V={V} {kind}")
    R = B * W
    assert tiles_of(R, V) >= 2
    x, scores, finished, eos = stream_inputs(shape, kind)
    want, gap = select_exactly(x, scores, W, finished, eos)
    err = U * sum_error(R, V)
    assert gap > 2 * err
    xd, sd, fd = dev(x), dev(scores), dev(finished)
    ws = torch.zeros(tb.bitnet_beam_select_workspace_bytes(B, W, V), dtype=torch.uint8, device="cuda:0")
    first = None
    for _ in range(2):
        out = [torch.empty(R, device="cuda:0")] + [
            torch.empty(R, dtype=torch.int32, device="cuda:0") for _ in range(3)]
        tb.bitnet_beam_select_into(B, W, V, xd, sd, fd, eos, *out, ws)
        got = [host(t) for t in out]
        for a, n in zip(got[1:], ("tokens", "parents", "finished")):
            assert np.array_equal(a, want[n]), n
        s, exact = got[0].astype(np.float64), want["scores"]
        inf = exact == -np.inf
        assert np.array_equal(s == -np.inf, inf)
        off = np.abs(s[~inf] - exact[~inf])
        assert (off <= U * np.abs(exact[~inf]) + err).all(), float(off.max() / U)
        assert first is None or first == got[0].tobytes()
        first = got[0].tobytes()
    say(f"  off by up to {float(off.max() / U):.1f} u of {err / U:.0f} + the rounding")


# ---- the largest sizes that are accepted ------------------------------------------

def test_select_of_the_largest_vocabulary(tb):  # noqa: F811
    """2^30 - 1 logits, rows 2^31 - 1 apart: 4096 tiles a thread."""
    import torch
    V, ld, W = (1 << 30) - 1, (1 << 31) - 1, 2
    say("[range] selection of 2^30 - 1 logits")
    x = torch.empty(ld + V, device="cuda:0")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(3)
    rows = [x[r * ld:r * ld + V] for r in range(W)]
    best = [[V - 1, 5, V // 2], [V // 3, V - 2, 0]]
    lse = []
    for row, b in zip(rows, best):
        for part in row.split(1 << 26):
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda:0"))
        row[torch.tensor(b, device="cuda:0")] = torch.tensor([9.0, 8.5, 8.0], device="cuda:0")
        total = sum(float(part.double().exp().sum()) for part in row.split(1 << 26))
        lse.append(np.log(total))
    scores = np.array([-1, -1.25], np.float32)
    cand = sorted((-(float(s) + v - e), b) for s, e, bs in zip(scores, lse, best)
                  for v, b in zip((9.0, 8.5, 8.0), bs))
    ws = torch.zeros(tb.bitnet_beam_select_workspace_bytes(1, W, V), dtype=torch.uint8, device="cuda:0")
    s = torch.empty(W, device="cuda:0")
    t, p = (torch.empty(W, dtype=torch.int32, device="cuda:0") for _ in range(2))
    tb.bitnet_beam_select_into(1, W, V, torch.as_strided(x, (W, V), (ld, 1)), dev(scores), None, 0,
                               s, t, p, None, ws)
    err = U * sum_error(W, V)
    assert host(t).tolist() == [b for _, b in cand[:W]]
    off = np.abs(host(s).astype(np.float64) - [-c for c, _ in cand[:W]])
    say(f"  off by up to {off.max() / U:.0f} u of {err / U:.0f}")
    assert (off <= U * 32 + err).all()
    assert [b in best[r] for r, b in zip(host(p).tolist(), host(t).tolist())] == [True] * W


def test_map_of_the_most_tokens(tb):  # noqa: F811
    """Room for 2^31 - 1 tokens, of which few are there: the rest is -1."""
    import torch
    T, B, ps, mp = (1 << 31) - 1, 3, 1024, 2
    say("[range] map of 2^31 - 1 tokens")
    pool, state = tb.KvPool.empty(B, mp, 8, ps)
    new = np.array([2000, 0, 1500], np.int32)
    out = tb.bitnet_kv_map(pool, T, dev(new), state)
    assert host(out["starts"]).tolist() == [0, 2000, 2000, 3500]
    want = np.concatenate([np.arange(2000), np.arange(1500)])
    assert np.array_equal(host(out["positions"][:3500]), want)
    slots = host(out["slots"][:3500])
    assert np.array_equal(slots, np.repeat(host(pool.tables)[[0, 2]], 1024, 1).reshape(-1)[
        np.concatenate([np.arange(2000), 2048 + np.arange(1500)])] * ps + want % ps)
    for n in ("slots", "positions", "rows"):
        for part in out[n][3500:].split(1 << 28):
            assert (part == -1).all().item(), n


def test_append_of_the_most_tokens(tb):  # noqa: F811
    import torch
    T, D, ps = (1 << 23) - 1, 64, 1024
    say("[range] append of 2^23 - 1 tokens")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(4)
    cache = tb.KvCache.empty(1, 1 << 13, 1, ps, D)
    slots = torch.randperm(1 << 23, generator=gen, device="cuda:0")[:T].int()
    slots[7] = -1
    k, v = (torch.randn(T, D, generator=gen, device="cuda:0") for _ in range(2))
    cache.k.zero_(), cache.v.zero_()
    tb.bitnet_kv_append(cache, 0, k, v, slots)
    for c, x in ((cache.k, k), (cache.v, v)):
        want = torch.zeros(1 << 23, D, dtype=torch.bfloat16, device="cuda:0")
        live = torch.arange(T, device="cuda:0") != 7
        want[slots[live].long()] = x[live].bfloat16()
        assert torch.equal(c.view(-1, D), want)


def test_reorder_of_the_most_rows_and_layers(tb):  # noqa: F811
    """4096 beams in 1024 layers, each beam's last page half filled."""
    import torch
    B, W, D, ps, layers = 128, 32, 64, 2, 1024
    say("[range] reordering of 4096 beams in 1024 layers")
    R = B * W
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(5)
    cache = tb.KvCache.empty(layers, 2 * R, 1, ps, D, torch.int8)
    for c in (cache.k, cache.v):
        c.copy_(torch.randint(-128, 128, c.shape, generator=gen, device="cuda:0", dtype=torch.int8))
    for c in (cache.k_scale, cache.v_scale):
        c.copy_(torch.rand(c.shape, generator=gen, device="cuda:0"))
    tables = torch.randperm(2 * R, generator=gen, device="cuda:0").int().view(R, 2)
    beam = torch.randint(0, W, (B, W), generator=gen, device="cuda:0")
    parents = (beam + W * torch.arange(B, device="cuda:0")[:, None]).reshape(-1).int()
    lens = torch.full((R,), 3, dtype=torch.int32, device="cuda:0")
    old = [c.clone() for c in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    out = tb.bitnet_beam_reorder(cache, tables, lens, parents, W)
    par, last = parents.long(), tables[:, 1].long()
    assert torch.equal(out[:, 0], tables[par, 0])
    assert torch.equal(out[:, 1].long().view(B, W).sort(1).values, last.view(B, W).sort(1).values)
    for c, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), old):
        new = out[:, 1].long()
        assert torch.equal(c[:, new, :, :1], o[:, last[par], :, :1])      # the token in use
        assert torch.equal(c[:, :, :, 1], o[:, :, :, 1])                  # the other place
        full = tables[:, 0].long()
        assert torch.equal(c[:, full], o[:, full])
