"""GPU parity of the cache and beam-search calls with their plain definitions
(oracle/decode_step.py, fp64), through the C ABI.

Whole numbers, pages, 8-bit codes and rotated rows are compared bit for bit.
The attention's tolerance is the bound of its fp32 arithmetic: with u = 2^-24,
a score is a sum of D products of exactly represented terms (relative error of
the split queries below 4u), so it is off by at most (D + 16) u S, with
S = max_j scale * sum_i |q_i k_ji|; that is the relative error of its
probability, twice over for numerator and denominator; the sums over n tokens
add n u each, the exponentials, rescalings, joins and the division 64 u in all:
    |out - exact| <= u (2 (D + 16) S + 2 n + 64) sum_j p_j |v_j|.
8-bit rows add one rounding per scale (inside the 64).  A probability (relative
to the row's largest, which is 1) below the smallest normal number of its format
is lost: 2^-126 in fp32 and bf16; 2^-38 for fp16 values, whose probabilities are
scaled by 2^14 against fp16's spacing of 2^-24, and for 8-bit ones, whose
probabilities carry their token's scale relative to a power of two at most twice
the largest.  Where the likely tokens' v are zero that is all that is left of an
element: each token adds up to that much times max |v|."""
import sys

import numpy as np
import pytest

from oracle import decode_step as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LOST = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -38, "int8": 2.0 ** -38}


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def tb():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ternary_weight_decoder_amd import binding
    binding.lib()
    return binding


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def host(t):
    return t.cpu().numpy()


# ---- page map -----------------------------------------------------------------

def map_inputs(seed, B, ps, mp, full, kind, free_part=1.0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, full + 1, B)
    new = np.ones(B, np.int64)
    if kind == "mixed":
        u = rng.random(B)
        new = rng.integers(0, full + 1, B)
        new[u < 0.3] = 1
        new[u < 0.2] = -rng.integers(1, 5, (u < 0.2).sum())
        new[u < 0.1] = 0
        lens[u > 0.8] = 0
    held = -(-lens // ps)
    P = B * mp
    order = rng.permutation(P)
    tables = order.reshape(B, mp).copy()
    free = np.full(P, -1)
    rest = order.reshape(B, mp)[np.arange(mp) >= held[:, None]]
    n = int(len(rest) * free_part)
    free[:n] = rest[:n]
    tables[np.arange(mp) >= held[:, None]] = -1
    i32 = lambda a: np.ascontiguousarray(a, np.int32)
    return (P, i32(new), i32(np.concatenate([lens, held, [n]])), i32(tables), i32(tables),
            i32(free))


def run_map(tb, P, ps, T, new, state, tables, owned, free, in_place=True):
    import torch
    B = len(new)
    td, od, fd = dev(tables), dev(owned), dev(free)
    pool = tb.KvPool(P, ps, td, od, fd)
    sin = dev(state)
    if in_place:
        out = tb.bitnet_kv_map(pool, T, dev(new), sin)
        got = {"state": host(sin)}
    else:
        sout = torch.full_like(sin, -77)
        names = {"starts": B + 1, "slots": T, "positions": T, "rows": T, "status": B}
        out = {n: torch.full((c + 8,), -77, dtype=torch.int32, device="cuda:0")
               for n, c in names.items()}
        tb.bitnet_kv_map_into(pool, T, dev(new), sin, sout, *out.values())
        for n, c in names.items():
            assert (out[n][c:] == -77).all().item(), "canary"
            out[n] = out[n][:c]
        assert np.array_equal(host(sin), state)
        got = {"state": host(sout)}
    got.update({n: host(t) for n, t in out.items()})
    got.update(tables=host(td), owned=host(od), free=host(fd))
    return got


@pytest.mark.parametrize("B,ps,mp,full,T,kind,part", [
    (1, 1, 4, 3, 1, "step", 1.0), (1, 64, 2, 64, 1, "step", 1.0), (16, 64, 32, 1800, 16, "step", 1.0),
    (63, 16, 8, 60, 500, "mixed", 1.0), (64, 8, 12, 40, 4000, "mixed", 0.05),
    (257, 4, 9, 17, 8192, "mixed", 0.3), (1025, 2, 20, 15, 8193, "mixed", 1.0),
    (4096, 16, 5, 33, 70001, "mixed", 0.5), (300, 1024, 2, 900, 100000, "mixed", 1.0),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_map(tb, B, ps, mp, full, T, kind, part, in_place):
    say(f"[map] B={B} ps={ps} mp={mp} T={T} {kind} {part} in_place={in_place}")
    P, new, state, tables, owned, free = map_inputs(B + ps + T, B, ps, mp, full, kind, part)
    want = ref.kv_map(ps, P, T, new, state, tables, owned, free)
    got = run_map(tb, P, ps, T, new, state, tables, owned, free, in_place)
    for n in want:
        assert np.array_equal(got[n], want[n]), n


def test_map_bad_device_values(tb):
    """Lengths, counts, the stack's height and pages out of their ranges, and
    additions that pass 32 bits: clamped or refused as the header says."""
    say("[map] bad device values")
    big = 2 ** 31 - 1
    P, ps, mp = 12, 4, 3
    new = np.array([big, 1, 2, -big - 1, 5, 3], np.int32)
    state = np.array([5, -9, big, 7, 0, 4] + [2, -3, 1, 900, 0, 3] + [big], np.int32)
    tables = np.full((6, mp), 99, np.int32)
    owned = np.arange(18, dtype=np.int32).reshape(6, mp) - 4
    free = np.arange(12, dtype=np.int32)[::-1].copy()
    want = ref.kv_map(ps, P, 20, new, state, tables, owned, free)
    got = run_map(tb, P, ps, 20, new, state, tables, owned, free)
    for n in want:
        assert np.array_equal(got[n], want[n]), n
    assert want["status"].tolist() == [1, 0, 1, 0, 0, 1]


def test_map_sequence_returns_every_page(tb):
    """Requests come and go over many steps; at the end every page is free once."""
    import torch
    say("[map] forty steps")
    rng = np.random.default_rng(3)
    pool, state = tb.KvPool.empty(24, 16, 200, 8, device="cuda:0")
    for step in range(40):
        new = rng.integers(-1, 30, 24).astype(np.int32)
        before = [host(t) for t in (state, pool.tables, pool.owned, pool.free_pages)]
        want = ref.kv_map(8, 200, 400, new, *before)
        out = tb.bitnet_kv_map(pool, 400, dev(new), state)
        got = dict({n: host(t) for n, t in out.items()}, state=host(state),
                   tables=host(pool.tables), owned=host(pool.owned), free=host(pool.free_pages))
        for n in want:
            assert np.array_equal(got[n], want[n]), (step, n)
        live = got["slots"][got["slots"] >= 0]
        assert len(set(live.tolist())) == len(live) == got["starts"][-1]
    tb.bitnet_kv_map(pool, 1, torch.full((24,), -1, dtype=torch.int32, device="cuda:0"), state)
    assert sorted(host(pool.free_pages).tolist()) == list(range(200))
    assert host(state).tolist() == [0] * 48 + [200]


# ---- append --------------------------------------------------------------------

def make_pages(seed, layers, pages, kv, ps, D, dtype, heads_first=True, gap=0):
    """Two cache tensors [layers, pages, kv, ps, D] of garbage (NaN for the float
    types) in strided memory, and their scales."""
    import torch
    out = []
    for _ in range(2):
        shape = (layers, pages, kv, ps, D + gap) if heads_first else (layers, pages, ps, kv, D + gap)
        if dtype is torch.int8:
            t = torch.full(shape, -128, dtype=dtype, device="cuda:0")
        else:
            t = torch.full(shape, float("nan"), dtype=dtype, device="cuda:0")
        out.append((t if heads_first else t.transpose(2, 3))[..., :D])
    if dtype is not torch.int8:
        return out + [None, None]
    return out + [torch.full((layers, pages, kv, ps), float("nan"), device="cuda:0")
                  for _ in range(2)]


def rope_tables(max_pos, D):
    ang = np.arange(max_pos)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}[name]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("T,kv,G,D,ps,hf,gap,rope,strided", [
    (1, 1, 1, 64, 1, True, 0, True, False), (3, 2, 6, 128, 16, False, 0, True, True),
    (65, 3, 5, 256, 8, True, 16, True, False), (7, 8, 1, 64, 1024, False, 32, False, True),
    (300, 2, 6, 128, 64, True, 0, True, True), (5, 1, 40, 128, 2, True, 0, True, False),
    (9, 5, 0, 128, 16, True, 0, True, False),
])
def test_append(tb, dt, T, kv, G, D, ps, hf, gap, rope, strided):
    import torch
    say(f"[append] {dt} T={T} kv={kv} G={G} D={D} ps={ps} hf={hf} rope={rope} strided={strided}")
    rng = np.random.default_rng(T * 7 + D)
    dtype, max_pos, layers = dtype_of(dt), 500, 2
    pages = -(-T // ps) + 2
    caches = make_pages(1, layers, pages, kv, ps, D, dtype, hf, gap)
    before = [None if c is None else c.clone() for c in caches]
    cache = tb.KvCache(*caches)
    H = kv * G
    scale = np.exp(rng.normal(0, 2, (T, 1)))
    q, k, v = ((rng.normal(0, 1, (T, n * D)) * scale).astype(np.float32) for n in (H, kv, kv))
    k[0, :D] = 0.0
    if T > 2:
        v[2, -D:] = 1e-45     # its 8-bit scale rounds to zero
    slots = rng.permutation(pages * ps)[:T].astype(np.int32)
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    skip = np.zeros(T, bool)
    if T > 4:                 # padding and bad values: skipped
        slots[1], slots[3] = -1, pages * ps
        skip[[1, 3]] = True
        if rope:
            pos[4] = max_pos
            skip[4] = True
    cos, sin = rope_tables(max_pos, D)

    def rows(a):
        t = dev(a)
        if strided:
            w = torch.full((T, a.shape[1] + 12), float("nan"), device="cuda:0")
            w[:, :a.shape[1]] = t
            t = w[:, :a.shape[1]]
        return t

    args = [rows(k), rows(v), dev(slots)] + ([dev(pos), dev(cos), dev(sin)] if rope else [])
    with_q = rope and G > 0
    got_q = tb.bitnet_kv_append(cache, 1, *args, **({"q": rows(q)} if with_q else {}))
    if rope:
        c, s = cos[np.minimum(pos, max_pos - 1)], sin[np.minimum(pos, max_pos - 1)]
        if with_q:
            want_q = ref.rotate(q.reshape(T, H, D), c, s).reshape(T, -1)
            want_q[skip] = 0.0
            assert host(got_q).tobytes() == want_q.tobytes()
        k = ref.rotate(k.reshape(T, kv, D), c, s)
    else:
        assert got_q is None
    for x, page_t, old, sc, old_sc in ((k, caches[0], before[0], caches[2], before[2]),
                                       (v, caches[1], before[1], caches[3], before[3])):
        x = x.reshape(T, kv, D)[~skip]
        at = slots[~skip].astype(np.int64)
        want = old.clone()
        if dt == "int8":
            codes, scales = ref.quant_rows(x)
            want[1, at // ps, :, at % ps] = dev(codes)
            want_sc = old_sc.clone()
            want_sc[1, at // ps, :, at % ps] = dev(scales)
            assert torch.equal(want_sc.view(torch.int32), sc.view(torch.int32))
            assert torch.equal(want, page_t)
        else:
            want[1, at // ps, :, at % ps] = dev(x).to(dtype)
            assert torch.equal(want.contiguous().view(torch.int16),
                               page_t.contiguous().view(torch.int16))
        whole = page_t._base if page_t._base is not None else page_t
        if gap:   # channels between the rows are left alone
            rest = whole[..., D:].float()
            assert (torch.isnan(rest) | (rest == -128)).all().item()


def test_append_in_place_queries_and_no_tokens(tb):
    import torch
    say("[append] q_out == q, and T = 0")
    T, kv, H, D = 6, 2, 4, 64
    cache = tb.KvCache(*make_pages(0, 1, 4, kv, 4, D, torch.bfloat16)[:2])
    rng = np.random.default_rng(0)
    q, k = (rng.normal(0, 1, (T, n * D)).astype(np.float32) for n in (H, kv))
    cos, sin = rope_tables(10, D)
    pos = np.arange(T, dtype=np.int32)
    qd = dev(q)
    tb.bitnet_kv_append_into(cache, 0, T, H, dev(k), dev(k), dev(pos), dev(pos), dev(cos), dev(sin),
                             qd, qd)
    assert host(qd).tobytes() == ref.rotate(q.reshape(T, H, D), cos[pos], sin[pos]).tobytes()
    e = torch.empty(0, kv * D, device="cuda:0")
    assert tb.bitnet_kv_append(cache, 0, e, e, torch.empty(0, dtype=torch.int32, device="cuda:0")) is None


# ---- attention -----------------------------------------------------------------

def attend_inputs(seed, lens, mp, kv, G, D, ps, dt, hf=True, gap=0, table_rows=None, spread=1.0):
    """Pages of garbage with the rows' tokens written in; returns device inputs
    and the fp64 values per row."""
    import torch
    rng = np.random.default_rng(seed)
    R = len(lens)
    P = sum(-(-n // ps) for n in lens) + 3
    caches = make_pages(seed, 2, P, kv, ps, D, dtype_of(dt), hf, gap)
    order = rng.permutation(P).astype(np.int32)
    tables = rng.choice(np.array([-1, P, 2 ** 31 - 1, -2 ** 31], np.int64), (R, mp)).astype(np.int32)
    ks, vs, used = [], [], 0
    for r, n in enumerate(lens):
        pages = order[used:used + -(-n // ps)]
        used += len(pages)
        tables[r, :len(pages)] = pages
        j = np.arange(n)
        vals = []
        for c, sc in ((caches[0], caches[2]), (caches[1], caches[3])):
            x = rng.normal(0, spread, (n, kv, D)).astype(np.float32)
            if dt == "int8":
                q, s = ref.quant_rows(x)
                sc[1, pages[j // ps], :, j % ps] = dev(s)
                c[1, pages[j // ps], :, j % ps] = dev(q)
                vals.append(q.astype(np.float64) * s[..., None])
            else:
                t = dev(x).to(c.dtype)
                c[1, pages[j // ps], :, j % ps] = t
                vals.append(host(t.double()))
        ks.append(vals[0].transpose(1, 0, 2))
        vs.append(vals[1].transpose(1, 0, 2))
    q = rng.normal(0, 1, (R, kv * G * D)).astype(np.float32)
    return caches, tables, q, ks, vs


def check_attention(out, lse, q, ks, vs, scale, D, lost=2.0 ** -126):
    H = q.shape[1] // D
    for t in range(q.shape[0]):
        n = ks[t].shape[1]
        o, l, smax, mag = ref.attention(q[t].reshape(H, D), ks[t], vs[t], scale)
        tol = U * (2 * (D + 16) * smax[:, None] + 2 * n + 64) * mag
        tol += n * lost * np.abs(vs[t]).max(initial=0.0)
        err = np.abs(out[t].reshape(H, D) - o)
        assert (err <= tol).all(), (t, n, float((err / np.maximum(tol, 1e-300)).max()))
        if n == 0:
            assert (out[t] == 0).all() and (lse[t] == -np.inf).all()
        else:
            bound = U * ((D + 16) * smax + n + 64 + 2 * np.abs(l))
            assert (np.abs(lse[t] - l) <= bound).all(), (t, n)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("lens,kv,G,D,ps,hf,gap", [
    ([1], 1, 1, 64, 16, True, 0),
    ([0, 1, 2, 31, 32, 33], 2, 6, 128, 16, True, 0),
    ([127, 128, 129, 0, 255, 257], 2, 3, 64, 8, False, 0),
    ([63, 64, 65, 500], 1, 16, 256, 64, False, 16),
    ([1000, 3], 1, 17, 128, 1, True, 0),
    ([77], 4, 1, 128, 2, True, 48),
    ([300, 20], 1, 64, 64, 32, True, 0),
    ([2049], 2, 6, 128, 1024, True, 0),
    ([1801, 225, 1000], 2, 6, 128, 64, False, 0),
])
def test_attention(tb, dt, lens, kv, G, D, ps, hf, gap):
    say(f"[attend] {dt} lens={lens} kv={kv} G={G} D={D} ps={ps} hf={hf} gap={gap}")
    mp = max(-(-max(lens) // ps), 1) + 2
    caches, tables, q, ks, vs = attend_inputs(len(lens) + D + ps, lens, mp, kv, G, D, ps, dt, hf, gap)
    cache = tb.KvCache(*caches)
    out, lse = tb.bitnet_paged_attention(cache, 1, dev(q), dev(tables),
                                         dev(np.array(lens, np.int32)), return_lse=True)
    check_attention(host(out), host(lse), q, ks, vs, D ** -0.5, D, LOST[dt])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("n,max_len", [(9000, 9000), (32767, 32768), (5, 32768), (20000, 131072)])
def test_attention_long(tb, dt, n, max_len):
    """One row, where the length is split, under bounds tight and loose."""
    say(f"[attend] long {dt} n={n} max_len={max_len}")
    D, ps, kv, G = 128, 64, 2, 6
    caches, tables, q, ks, vs = attend_inputs(n, [n], max_len // ps + 1, kv, G, D, ps, dt)
    cache = tb.KvCache(*caches)
    out, lse = tb.bitnet_paged_attention(cache, 1, dev(q), dev(tables), dev(np.array([n], np.int32)),
                                         max_len, 0.1, return_lse=True)
    check_attention(host(out), host(lse), q, ks, vs, 0.1, D, LOST[dt])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
def test_attention_large_scores(tb, dt):
    """Scores of hundreds: the softmax is almost one-hot, its maximum moves from
    tile to tile, and most exponentials underflow."""
    say(f"[attend] large scores {dt}")
    lens, kv, G, D, ps = [700, 64, 1500], 2, 4, 128, 16
    caches, tables, q, ks, vs = attend_inputs(5, lens, 100, kv, G, D, ps, dt, spread=12.0)
    q *= 5
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables),
                                         dev(np.array(lens, np.int32)), scale=1.0, return_lse=True)
    check_attention(host(out), host(lse), q, ks, vs, 1.0, D, LOST[dt])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
def test_attention_small_values_and_uneven_channels(tb, dt):
    """Keys and values down in fp16's subnormal numbers, queries with channels a
    million times others, 8-bit scales that differ by many powers of two."""
    say(f"[attend] small values {dt}")
    lens, kv, G, D, ps = [130, 65], 2, 3, 128, 16
    for spread, qs in ((2e-6, 1e6), (1.0, 1.0), (3e3, 1e-3)):
        caches, tables, q, ks, vs = attend_inputs(8, lens, 12, kv, G, D, ps, dt, spread=spread)
        q *= qs
        q[:, ::7] *= 1e-6
        if dt == "int8":
            rng = np.random.default_rng(1)
            for sc, vals in ((caches[2], ks), (caches[3], vs)):
                f = np.exp2(rng.integers(-30, 1, tuple(sc.shape[1:]))).astype(np.float32)
                sc[1] *= dev(f)
                for r, n in enumerate(lens):
                    j = np.arange(n)
                    vals[r] *= f[tables[r, j // ps], :, j % ps].T[..., None]
        out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables),
                                             dev(np.array(lens, np.int32)), scale=0.3,
                                             return_lse=True)
        check_attention(host(out), host(lse), q, ks, vs, 0.3, D, LOST[dt])


def test_attention_rows_lens_and_bad_pages(tb):
    """Several queries of one request (each with its own length), requests out
    of range, lengths below 0 and above max_len, pages out of range inside the
    length, strided queries: the rows are those of the tokens that are left."""
    import torch
    say("[attend] rows, lens out of range, bad pages")
    lens, kv, G, D, ps, mp = [200, 90], 2, 2, 64, 16, 20
    for dt in ("bf16", "fp16", "int8"):
        caches, tables, q0, ks, vs = attend_inputs(11, lens, mp, kv, G, D, ps, dt)
        tables[1, 2], tables[1, 4] = -5, 2 ** 30          # tokens 32-47 and 64-79
        rows = np.array([0, 0, 0, 1, 1, 2, -1, 0], np.int32)
        want = [200, 1, 130, 90, 40, 50, 50, 0]
        ll = np.array([200, 1, 130, 90, 40, 50, 50, -3], np.int32)
        H = kv * G
        q = np.random.default_rng(1).normal(0, 1, (8, H * D)).astype(np.float32)
        kk, vv = [], []
        for r, n in zip(rows, want):
            if not 0 <= r < 2:
                n, r = 0, 0
            keep = np.arange(n)
            if r == 1:
                keep = keep[(keep // 16 != 2) & (keep // 16 != 4)]
            kk.append(ks[r][:, keep])
            vv.append(vs[r][:, keep])
        wide = torch.full((8, H * D + 20), float("nan"), device="cuda:0")
        wide[:, :H * D] = dev(q)
        out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, wide[:, :H * D], dev(tables),
                                             dev(ll), rows=dev(rows), return_lse=True)
        check_attention(host(out), host(lse), q, kk, vv, D ** -0.5, D, LOST[dt])
        # above max_len: clamped to it
        out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q[:1]), dev(tables),
                                             dev(np.array([10 ** 9], np.int32)), max_len=150,
                                             return_lse=True)
        check_attention(host(out), host(lse), q[:1], [ks[0][:, :150]], [vs[0][:, :150]], D ** -0.5,
                        D, LOST[dt])


def test_attention_shapes_follow_each_other_on_one_workspace(tb):
    """One zeroed workspace serves calls of different shapes in turn; repeated
    calls give the same bits."""
    import torch
    say("[attend] one workspace, many shapes")
    shapes = [([4000], 2, 6, 128, 64), ([100, 3000, 0, 7], 1, 3, 64, 16), ([4000], 2, 6, 128, 64),
              ([900] * 9, 4, 2, 64, 8), ([2500, 2500], 1, 40, 256, 32)]
    sets = []
    need = 0
    for i, (lens, kv, G, D, ps) in enumerate(shapes):
        mp = -(-max(lens) // ps)
        sets.append(attend_inputs(i, lens, mp, kv, G, D, ps, "bf16"))
        need = max(need, tb.bitnet_paged_attention_workspace_bytes(len(lens), kv * G, kv, D, mp * ps))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda:0")
    first = {}
    for turn in range(3):
        for i, (lens, kv, G, D, ps) in enumerate(shapes):
            caches, tables, q, ks, vs = sets[i]
            out = torch.full((len(lens) + 1, kv * G * D), float("nan"), device="cuda:0")
            lse = torch.empty(len(lens), kv * G, device="cuda:0")
            tb.bitnet_paged_attention_into(tb.KvCache(*caches), 1, len(lens), kv * G, dev(q),
                                           dev(tables), dev(np.array(lens, np.int32)),
                                           tables.shape[1] * ps, 0.1, out, ws, lse=lse)
            assert torch.isnan(out[-1]).all().item(), "canary"
            check_attention(host(out[:-1]), host(lse), q, ks, vs, 0.1, D)
            assert first.setdefault(i, host(out[:-1]).tobytes()) == host(out[:-1]).tobytes()


# ---- beam selection --------------------------------------------------------------

def check_select(tb, x, scores, W, finished=None, eos=-1, ld=None, exact_ties=False):
    import torch
    R, V = x.shape
    xd = dev(x)
    if ld:
        wide = torch.full((R, ld), float("inf"), device="cuda:0")
        wide[:, :V] = xd
        xd = wide[:, :V]
    want = ref.beam_select(x, scores, W, finished, eos)
    # The selection is decided where no two beams' scores meet within the error
    # of their sums of exp: 8 u for the sum over lanes and waves, one u for each
    # further logit of a thread (V / 256, at most 16), 2 u for exp and at most
    # 14 u for its argument's rounding (logits that are 14 or more below the
    # largest weigh nothing), twice.
    assert want["gap"] > 2 * U * (24 + min(16, -(-V // 256))) or exact_ties
    out = tb.bitnet_beam_select(xd, dev(scores), W, None if finished is None else dev(finished), eos)
    for n in ("tokens", "parents") + (("finished",) if finished is not None else ()):
        assert np.array_equal(host(out[n]), want[n]), n
    got, exact = host(out["scores"]).astype(np.float64), want["scores"]
    inf = exact == -np.inf
    assert np.array_equal(got == -np.inf, inf)
    # one fp32 rounding, and 64 u for the fp32 terms of the sum of exp
    assert (np.abs(got - exact)[~inf] <= U * (np.abs(exact[~inf]) + 64)).all()
    return out


def logits(seed, R, V, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (R, V)).astype(np.float32)
    x[:, rng.integers(0, V, max(V // 10, 1))] = -np.inf
    return x, (-5 - 3 * rng.random(R)).astype(np.float32)


@pytest.mark.parametrize("B,W,V", [(1, 1, 1), (1, 1, 151936), (1, 4, 151936), (4, 4, 151936),
                                   (3, 5, 1000), (2, 32, 33), (1, 32, 70001), (2, 2, 4095),
                                   (2, 2, 4096), (2, 3, 4097), (1, 8, 8200), (40, 1, 5000),
                                   (128, 32, 37), (5, 7, 16385), (16, 16, 20000)])
def test_select(tb, B, W, V):
    say(f"[select] B={B} W={W} V={V}")
    x, s = logits(B * 1000 + W + V, B * W, V)
    check_select(tb, x, s, W, ld=V + 3 if V < 10000 else None)


@pytest.mark.parametrize("W,V", [(1, 500), (4, 5000), (6, 151936), (32, 40)])
def test_select_finished_beams(tb, W, V):
    say(f"[select] finished W={W} V={V}")
    for eos in (0, V - 1, V // 2):
        x, s = logits(W + V + eos, 3 * W, V)
        rng = np.random.default_rng(eos)
        fin = (rng.random(3 * W) < 0.4).astype(np.int32) * 7
        fin[:W] = 1                       # a whole group has ended
        x[W:, eos] = 9.0
        check_select(tb, x, s, W, fin, eos)


def test_select_ties_and_special_values(tb):
    """Equal logits go to the lower token, equal beams to the lower beam; -inf,
    NaN, +inf, rows without a token, dead beams, both zeros."""
    say("[select] ties and special values")
    for V in (50, 9000):
        x = np.zeros((4, V), np.float32)
        check_select(tb, x, np.full(4, -1, np.float32), 4, exact_ties=True)
        x[:, ::2] = -0.0
        check_select(tb, x, np.array([-1, -1, -2, -2], np.float32), 2, exact_ties=True)
        x, s = logits(V, 4, V)
        x[1] = x[0]
        s[1] = s[0]
        check_select(tb, x, s, 4, exact_ties=True)
        x[0], s[2] = -np.inf, -np.inf       # nothing to take; a dead beam
        x[1, 3], x[1, 4], x[3, V - 1] = np.nan, np.inf, np.nan
        check_select(tb, x, s, 4)
        x[:] = -np.inf                      # only tokens that cannot be taken
        check_select(tb, x, s, 4, exact_ties=True)
        s[:] = -np.inf
        x, _ = logits(V + 1, 4, V)
        check_select(tb, x, s, 4, exact_ties=True)
        s[:] = [np.nan, np.inf, -1, -2]
        check_select(tb, x, s, 4)
        # sorted logits: all of a chunk's largest sit next to each other
        for sign in (1, -1):
            x = np.tile((sign * np.arange(V) * 1e-3).astype(np.float32), (4, 1))
            check_select(tb, x, np.array([-1, -9, -17, -25], np.float32), 4)
        # the greatest and smallest finite logits
        x, s = logits(V + 2, 2, V)
        x[0, 1], x[1, :] = 3e38, -3e38
        check_select(tb, x, s, 2, exact_ties=True)


@pytest.mark.parametrize("W,V", [(32, 40), (32, 20000), (4, 151936), (8, 151936), (5, 151936)])
def test_select_everything_ties(tb, W, V):
    """All candidates of a group equal, alive or dead; and rising logits, where
    every tile of a row replaces what the ones before it gave."""
    say(f"[select] ties W={W} V={V}")
    x = np.zeros((W, V), np.float32)
    check_select(tb, x, np.full(W, -1, np.float32), W, exact_ties=True)
    check_select(tb, x, np.full(W, -np.inf, np.float32), W, exact_ties=True)
    check_select(tb, x, np.full(W, -1, np.float32), W, (np.arange(W) % 2).astype(np.int32), V - 1,
                 exact_ties=True)
    x[:] = (np.arange(V) * 1e-3).astype(np.float32)
    check_select(tb, x, -np.arange(W, dtype=np.float32) * 0.25, W, exact_ties=True)


def test_select_in_place(tb):
    import torch
    say("[select] scores and flags in place, one workspace for many shapes")
    ws = torch.zeros(tb.bitnet_beam_select_workspace_bytes(4, 8, 30000), dtype=torch.uint8,
                     device="cuda:0")
    for turn, (B, W, V) in enumerate([(4, 8, 30000), (1, 3, 100), (4, 8, 30000), (2, 2, 9000)] * 2):
        x, s = logits(turn, B * W, V)
        fin = (np.arange(B * W) % 3 == 0).astype(np.int32)
        want = ref.beam_select(x, s, W, fin, 2)
        assert want["gap"] > 1e-5
        sd, fd = dev(s), dev(fin)
        t, p = (torch.full((B * W + 4,), -7, dtype=torch.int32, device="cuda:0") for _ in range(2))
        tb.bitnet_beam_select_into(B, W, V, dev(x), sd, fd, 2, sd, t, p, fd, ws)
        assert (t[-4:] == -7).all().item() and (p[-4:] == -7).all().item()
        assert np.array_equal(host(t)[:-4], want["tokens"])
        assert np.array_equal(host(p)[:-4], want["parents"])
        assert np.array_equal(host(fd), want["finished"])
        np.testing.assert_allclose(host(sd), want["scores"], rtol=U * 66, atol=U * 64)


# ---- beam reordering ---------------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "int8"])
@pytest.mark.parametrize("B,W,ps,length,layers,kv,D,hf", [
    (1, 1, 16, 5, 1, 1, 64, True), (2, 4, 16, 37, 3, 2, 128, False), (3, 5, 64, 1, 1, 2, 64, True),
    (1, 32, 8, 23, 2, 1, 256, True), (2, 4, 16, 32, 2, 2, 64, True), (1, 3, 1, 6, 2, 2, 64, True),
    (2, 8, 128, 127, 2, 3, 64, False), (2, 2, 16, 0, 1, 1, 64, True),
])
def test_reorder(tb, dt, B, W, ps, length, layers, kv, D, hf):
    import torch
    say(f"[reorder] {dt} B={B} W={W} ps={ps} length={length} layers={layers}")
    rng = np.random.default_rng(B + W + ps + length)
    R, mp = B * W, length // ps + 3
    shared = length // ps
    P = R * mp + 2
    tables = rng.permutation(P)[:R * mp].reshape(R, mp).astype(np.int32)
    for g in range(0, R, W):
        tables[g:g + W, :shared] = tables[g, :shared]
    caches = [c for c in make_pages(0, layers, P, kv, ps, D, dtype_of(dt), hf)]
    for c in caches:
        if c is not None and c.dtype is torch.int8:
            c.copy_(torch.randint(-128, 128, c.shape, device="cuda:0", dtype=torch.int8))
        elif c is not None:
            c.copy_(torch.randn(c.shape, device="cuda:0"))
    bits = (lambda t: None if t is None else
            host(t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])))
    parents = rng.integers(0, W, R)
    parents[:W] = W - 1 if W > 1 else 0
    if R > 5:
        parents[R - 1] = -3 * W                  # not of the group: the row itself
    parents = (parents + np.repeat(np.arange(B) * W, W)).astype(np.int32)
    lens = np.full(R, length, np.int32)
    want = ref.beam_reorder(*[bits(c) for c in caches], W, parents, lens, tables)
    td = dev(tables)
    out = tb.bitnet_beam_reorder(tb.KvCache(*caches), td, dev(lens), dev(parents), W)
    assert np.array_equal(host(out), want[-1]) and np.array_equal(host(td), tables)
    for c, w in zip(caches, want):
        assert c is None or np.array_equal(bits(c), w)


def test_reorder_bad_device_values(tb):
    """Pages out of range are not copied, lengths are clamped."""
    import torch
    say("[reorder] bad pages and lengths")
    c = [torch.randn(1, 9, 1, 4, 64, device="cuda:0").to(torch.bfloat16) for _ in range(2)]
    for tables, length in (([[0, -1], [2, 3]], 6), ([[0, 1], [2, 9]], 6), ([[0, 1], [2, 3]], 2 ** 31 - 1),
                           ([[0, 1], [2, 3]], -5)):
        tables = np.array(tables, np.int32)
        before = [t.clone() for t in c]
        par = np.zeros(2, np.int32)
        want = ref.beam_reorder(host(c[0].view(torch.int16)), host(c[1].view(torch.int16)), None, None,
                                2, par, [length] * 2, tables)
        out = tb.bitnet_beam_reorder(tb.KvCache(*c), dev(tables), dev(np.full(2, length, np.int32)),
                                     dev(par), 2)
        assert np.array_equal(host(out), want[-1])
        assert all(torch.equal(a, b) for a, b in zip(c, before))
