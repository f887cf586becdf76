"""GPU parity of the calls around a prompt's projections with their plain
definitions (oracle/prompt.py, fp64), through the C ABI.

Chunk attention: the tolerance of the attention of single tokens, which has the
same arithmetic (fp32 sums of exactly multiplied 16-bit terms): with u = 2^-24,
S = max_j scale * sum_i |q_i k_ji| and n tokens,
    |out - exact| <= u (2 (D + 16) S + 2 n + 64) sum_j p_j |v_j| + n LOST max |v|,
    |lse - exact| <= u ((D + 16) S + n + 64) + n LOST + u |lse|,
LOST what a probability (relative to the largest) loses below its format's
smallest numbers: 2^-126 for bf16; fp16 terms are sums down to 2^-24, half of which
is lost, of probabilities that are scaled to 2^9 or more at the largest, so 2^-34;
with 8-bit values a token's scale relative to a power of two at most twice the
largest one comes with it, so 2^-33.  lse is rounded once, and what its logarithm (2 u in units of
log 2, at most 24 of them) adds lies in the 64.

Norm and gated activation: fp64, rounded once: |y - exact| <= (1/2 ulp) (1 +
2^-20); below the normal numbers half of 2^-149.  8-bit rows are compared bit for
bit with the quantization of the call's own fp32 row.

Log probabilities: as the header says, e = (15 + 4 n + 2 ln V) u for lse and for
the sum that the entropy H divides by; the sum of e d, all of one sign, has the
same relative error and two roundings a term more, so H = log S - (sum e d) / S
is off by at most e + (2 e + 4 u) H, and u H for its own rounding."""
import math

import numpy as np
import pytest

from oracle import prompt as ref
from tests.test_gpu_decode_step import U, dev, host, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu
LOST = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -34, "int8": 2.0 ** -33}


# ---- chunk attention ------------------------------------------------------------

class Paged:
    """A cache of one or more layers with requests of given lengths in shuffled
    pages, and its values in fp64."""

    def __init__(self, tb, rng, dtype, lens, KV, D, PS, heads_first=True, layers=1, layer=0,
                 spare_pages=3, mp=None):
        import torch
        self.layer, self.KV, self.D, self.PS, self.dtype = layer, KV, D, PS, dtype
        R = len(lens)
        need = [-(-max(int(n), 0) // PS) for n in lens]
        self.mp = mp or max(need + [1]) + 1
        P = sum(need) + spare_pages
        shape = (layers, P, KV, PS, D) if heads_first else (layers, P, PS, KV, D)
        if dtype == "int8":
            k, v = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
            self.ks, self.vs = ((rng.random((layers, P, KV, PS)) * 0.05 + 0.001).astype(np.float32)
                                for _ in range(2))
        else:
            k, v = (rng.normal(0, 1, shape).astype(np.float32) for _ in range(2))
            self.ks = self.vs = None
        td = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}[dtype]
        self.kd, self.vd = (torch.from_numpy(x).to(td).to("cuda:0") for x in (k, v))
        if not heads_first:
            self.kd, self.vd = self.kd.transpose(2, 3), self.vd.transpose(2, 3)
        self.ksd, self.vsd = (None, None) if self.ks is None else (dev(self.ks), dev(self.vs))
        self.tables = np.full((R, self.mp), -7, np.int64)
        order, at = rng.permutation(P), 0
        for r, n in enumerate(need):
            self.tables[r, :n] = order[at:at + n]
            at += n
        self.P = P
        self.make(tb)

    def make(self, tb):
        self.cache = tb.KvCache(self.kd, self.vd, self.ksd, self.vsd)
        self.k, self.v = (t[self.layer].double().cpu().numpy() for t in (self.kd, self.vd))
        if self.ks is not None:
            self.k = self.k * self.ks[self.layer][..., None].astype(np.float64)
            self.v = self.v * self.vs[self.layer][..., None].astype(np.float64)

    def rows(self, x, r, n):
        t = np.arange(n)
        page = self.tables[r][t // self.PS] if n else np.zeros(0, int)
        there = (page >= 0) & (page < self.P)
        return x[page[there], :, t[there] % self.PS].transpose(1, 0, 2)

    def check(self, q, starts, lens, max_len, scale, out, lse):
        got = ref.chunk_attention(q, starts, lens, max_len, lambda r, n: self.rows(self.k, r, n),
                                  lambda r, n: self.rows(self.v, r, n), scale)
        D, worst = self.D, 0.0
        vmax = np.abs(self.v).max()
        for t, (want, want_lse, smax, mag, n) in got.items():
            tol = U * (2 * (D + 16) * smax + 2 * n + 64)[:, None] * mag + n * LOST[self.dtype] * vmax
            err = np.abs(out[t].astype(np.float64) - want)
            assert (err <= tol).all(), (t, n, (err / np.maximum(tol, 1e-300)).max())
            worst = max(worst, (err / np.maximum(tol, 1e-300)).max())
            none = np.isinf(want_lse)
            assert (np.isneginf(lse[t]) == none).all(), t
            ltol = U * ((D + 16) * smax + n + 64) + n * LOST[self.dtype]
            ok = np.abs(lse[t] - np.where(none, 0, want_lse)) <= ltol + U * np.abs(np.where(none, 0, want_lse))
            assert (ok | none).all(), t
        say(f"  worst error {worst:.2f} of the tolerance")
        return set(got)


def run_chunk(tb, pg, q, starts, lens, H, scale=None, max_len=None, pad=8, stride=None, ws=None):
    """The call with canaries around its outputs -> out [T, H, D], lse [T, H]."""
    import torch
    T, D = q.shape[0], pg.D
    scale = D ** -0.5 if scale is None else scale
    max_len = max_len or pg.mp * pg.PS
    R = len(lens)
    if stride:
        buf = torch.full((T, stride), float("nan"), device="cuda:0")
        buf[:, :H * D] = dev(q.reshape(T, -1))
        qd = buf[:, :H * D]
    else:
        qd = dev(q.reshape(T, -1))
    out = torch.full((T + pad, H * D), -77.0, device="cuda:0")
    lse = torch.full((T + pad, H), -77.0, device="cuda:0")
    n = tb.bitnet_chunk_attention_workspace_bytes(T, R, H, pg.KV, D, max_len)
    if ws is None:
        ws = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda:0")
    i32 = lambda a: dev(np.asarray(a, np.int64).astype(np.int32))
    for _ in range(2):   # the second call finds what the first left
        tb.bitnet_chunk_attention_into(pg.cache, pg.layer, T, H, qd, i32(starts), i32(lens),
                                       i32(pg.tables), max_len, scale, out, ws[:n], lse)
    assert (ws[n:] == 0xAB).all().item(), "behind the workspace"
    o, l = host(out), host(lse)
    assert (o[T:] == -77).all() and (l[T:] == -77).all(), "behind the outputs"
    rows = pg.check(q, starts, lens, max_len, scale, o[:T].reshape(T, H, D), l[:T])
    for t in set(range(T)) - rows:
        assert (o[t] == -77).all() and (l[t] == -77).all(), ("not a request's", t)
    return o[:T].reshape(T, H, D), l[:T]


def chunk_case(tb, seed, dtype, new, old, KV, G, D, PS, **kw):
    rng = np.random.default_rng(seed)
    new, old = np.asarray(new), np.asarray(old)
    opts = {n: kw.pop(n) for n in ("heads_first", "layers", "layer", "mp") if n in kw}
    pg = Paged(tb, rng, dtype, new + old, KV, D, PS, **opts)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.normal(0, 1, (int(starts[-1]) + kw.pop("behind", 0), KV * G, D)).astype(np.float32)
    return run_chunk(tb, pg, q, starts, new + old, KV * G, **kw)


SIZES = [
    # new, old, KV, G, PS
    ([1], [0], 1, 1, 8), ([1], [256], 2, 6, 64), ([4], [253], 2, 6, 64), ([33], [0], 2, 6, 16),
    ([22], [31], 1, 6, 32), ([128], [128], 1, 1, 64), ([129], [5], 2, 1, 1),
    ([0, 3, 0, 40, 1, 0], [7, 0, 0, 50, 200, 31], 2, 5, 16), ([5, 70, 1], [1000, 3, 64], 3, 16, 128),
    ([2, 9], [300, 0], 1, 64, 16), ([7, 7, 7, 7], [0, 1, 30, 33], 4, 7, 1024),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_chunk(tb, dtype, D, size):
    new, old, KV, G, PS = SIZES[size]
    say(f"[chunk] {dtype} D={D} new={new} old={old} KV={KV} G={G} PS={PS}")
    chunk_case(tb, size * 10 + D, dtype, new, old, KV, G, D, PS, heads_first=size % 2 == 0,
               behind=size % 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "int8"])
def test_chunk_prompt_and_long(tb, dtype):
    """A prompt whose items are cut into parts, and a piece far into a context."""
    say(f"[chunk] prompt of 700, {dtype}")
    chunk_case(tb, 1, dtype, [700], [0], 2, 6, 128, 16)
    say(f"[chunk] 40 at 6000, {dtype}")
    chunk_case(tb, 2, dtype, [40], [6000], 2, 6, 128, 64, heads_first=False)


@pytest.mark.parametrize("D", [64, 256])
def test_chunk_long_other_dims(tb, D):
    for dtype in ("bf16", "fp16", "int8"):
        say(f"[chunk] 30 at 3000, {dtype}, D={D}")
        chunk_case(tb, D, dtype, [30, 1], [3000, 900], 1, 8, D, 32)


def test_chunk_layers_strides_scale(tb):
    for dtype in ("bf16", "int8"):
        say(f"[chunk] layer 2 of 3, strided q, scale -0.3, bound below the table, {dtype}")
        chunk_case(tb, 5, dtype, [50, 3], [20, 90], 2, 3, 64, 16, layers=3, layer=2,
                   stride=6 * 64 + 20, scale=-0.3, max_len=96)


@pytest.mark.parametrize("R", [65, 300, 1000, 4096])
def test_chunk_many_requests(tb, R):
    say(f"[chunk] {R} requests")
    rng = np.random.default_rng(R)
    new = rng.integers(0, 3, R)
    new[R // 2] = 37
    chunk_case(tb, R, "fp16", new, rng.integers(0, 20, R), 1, 2, 64, 16)


def test_chunk_device_values_out_of_range(tb):
    """Starts that fall or leave [0, T], lengths out of range or shorter than
    what is new, pages out of range."""
    rng = np.random.default_rng(3)
    for dtype in ("bf16", "fp16", "int8"):
        say(f"[chunk] device values out of range, {dtype}")
        pg = Paged(tb, rng, dtype, [60, 90, 40, 70, 64, 33], 2, 64, 16)
        pg.tables[1, 2] = pg.P
        pg.tables[1, 3] = -1
        pg.tables[3, 0] = 2 ** 31 - 1
        pg.tables[4, :] = -5
        T, H = 100, 6
        q = rng.normal(0, 1, (T, H, 64)).astype(np.float32)
        mx = pg.mp * pg.PS
        lens = [10, 90, 2 ** 31 - 1, -5, 64, 33]
        pg.tables[2, :] = np.arange(pg.mp) % pg.P
        run_chunk(tb, pg, q, [5, 30, 30, 50, 40, 70, 95], lens, H)
        run_chunk(tb, pg, q, [-9, 30, 20, 2 ** 31 - 1, 0, 70, -1], lens, H)
        run_chunk(tb, pg, q, [200, 0, 0, 0, 0, 0, 0], lens, H)
        run_chunk(tb, pg, q, [0, 20, 40, 60, 80, 90, 100], [mx] * 6, H)


def test_chunk_is_causal(tb):
    """What a token holds reaches no row before it: infinities, NaN and huge
    scales in later tokens, and behind the last, change not a bit of them."""
    import torch
    rng = np.random.default_rng(4)
    for dtype in ("bf16", "fp16", "int8"):
        for n, old, at in ((40, 20, 43), (100, 0, 64), (30, 500, 517)):
            say(f"[causal] {dtype} {n} new after {old}, spoiled from {at}")
            pg = Paged(tb, rng, dtype, [n + old], 2, 128, 16)
            q = rng.normal(0, 1, (n, 4, 128)).astype(np.float32)
            a, la = run_chunk(tb, pg, q, [0, n], [n + old], 4)
            for bad in (float("nan"), float("inf"), -float("inf"), 1e30):
                for t in range(at, -(-(n + old) // 16) * 16):
                    page = int(pg.tables[0, t // 16])
                    for x, s in ((pg.kd, pg.ksd), (pg.vd, pg.vsd)):
                        if dtype == "int8":
                            s[0, page, :, t % 16] = abs(bad)
                        else:
                            x[0, page, :, t % 16] = bad
                out, lse = tb.bitnet_chunk_attention(
                    pg.cache, 0, dev(q.reshape(n, -1)), dev(np.array([0, n], np.int32)),
                    dev(np.array([n + old], np.int32)), dev(pg.tables.astype(np.int32)),
                    return_lse=True)
                seen = at - old   # rows that see none of it
                assert np.array_equal(host(out).reshape(a.shape)[:seen], a[:seen]), bad
                assert np.array_equal(host(lse)[:seen], la[:seen]), bad


def test_chunk_rows_with_bad_queries(tb):
    """A row with NaN or infinities leaves the others alone."""
    rng = np.random.default_rng(6)
    for dtype in ("bf16", "fp16", "int8"):
        say(f"[chunk] bad queries, {dtype}")
        pg = Paged(tb, rng, dtype, [90], 2, 64, 16)
        q = rng.normal(0, 1, (60, 6, 64)).astype(np.float32)
        a, la = run_chunk(tb, pg, q, [0, 60], [90], 6)
        bad = q.copy()
        bad[7, 2, 5], bad[30, 0, :], bad[31, 5, 63] = np.nan, np.inf, -np.inf
        out, lse = tb.bitnet_chunk_attention(
            pg.cache, 0, dev(bad.reshape(60, -1)), dev(np.array([0, 60], np.int32)),
            dev(np.array([90], np.int32)), dev(pg.tables.astype(np.int32)), return_lse=True)
        o, l = host(out).reshape(a.shape), host(lse)
        same = np.ones((60, 6), bool)
        same[7, 2] = same[30, 0] = same[31, 5] = False
        assert np.array_equal(o[same], a[same]) and np.array_equal(l[same], la[same])


def test_chunk_magnitudes(tb):
    """Large and small queries, keys and values, and outlier channels."""
    rng = np.random.default_rng(7)
    import torch
    for dtype in ("bf16", "fp16"):
        for qs, ks, vs in ((1e-6, 1.0, 1.0), (30.0, 5.0, 1e-3), (1e4, 1e-3, 1e3), (1.0, 1e-4, 1e-4)):
            say(f"[chunk] magnitudes {dtype} {qs} {ks} {vs}")
            pg = Paged(tb, rng, dtype, [150], 1, 128, 32)
            pg.kd *= ks
            pg.vd *= vs
            pg.kd[..., 5] *= 20
            pg.make(tb)
            q = (rng.normal(0, 1, (60, 4, 128)) * qs).astype(np.float32)
            run_chunk(tb, pg, q, [0, 60], [150], 4)


def test_chunk_equals_single_tokens(tb):
    """Beside the attention of single tokens, on the same cache and rows."""
    rng = np.random.default_rng(8)
    for dtype in ("bf16", "fp16", "int8"):
        say(f"[chunk] beside single tokens, {dtype}")
        new, old = np.array([3, 60, 1]), np.array([400, 10, 77])
        pg = Paged(tb, rng, dtype, new + old, 2, 128, 16)
        starts = np.r_[0, np.cumsum(new)]
        q = rng.normal(0, 1, (64, 12, 128)).astype(np.float32)
        a, la = run_chunk(tb, pg, q, starts, new + old, 12)
        rows = np.repeat(np.arange(3), new).astype(np.int32)
        lens = np.concatenate([o + 1 + np.arange(n) for o, n in zip(old, new)]).astype(np.int32)
        b, lb = tb.bitnet_paged_attention(pg.cache, 0, dev(q.reshape(64, -1)),
                                          dev(pg.tables.astype(np.int32)), dev(lens),
                                          rows=dev(rows), return_lse=True)
        assert np.abs(host(b).reshape(a.shape) - a).max() < 2e-5
        assert np.abs(host(lb) - la).max() < 2e-5


def test_chunk_one_workspace_for_all_shapes(tb):
    """Calls of different shapes follow each other on one workspace."""
    import torch
    rng = np.random.default_rng(9)
    ws = torch.full((80 << 20,), 0xAB, dtype=torch.uint8, device="cuda:0")
    for dtype, D, new, old in (("bf16", 128, [4], [800]), ("int8", 64, [90, 2], [0, 400]),
                               ("fp16", 256, [20], [600]), ("fp16", 128, [300], [0])):
        say(f"[chunk] shared workspace {dtype} {D}")
        new, old = np.array(new), np.array(old)
        pg = Paged(tb, rng, dtype, new + old, 2, D, 16)
        q = rng.normal(0, 1, (int(new.sum()), 8, D)).astype(np.float32)
        run_chunk(tb, pg, q, np.r_[0, np.cumsum(new)], new + old, 8, ws=ws)


# ---- rows ------------------------------------------------------------------------

def near(got, want):
    """fp32 values that are fp64 values rounded once."""
    want = np.asarray(want, np.float64)
    tol = np.abs(want) * 2.0 ** -24 * (1 + 2.0 ** -20) + 2.0 ** -150
    return (np.abs(got.astype(np.float64) - want) <= tol).all()


ROW_SIZES = [(1, 4), (1, 1536), (3, 64), (16, 1536), (5, 100), (17, 2048), (7, 2052), (16, 8960),
             (3, 10240), (2, 10244), (1, 32768), (1030, 1536), (1025, 260), (33, 8960), (260, 2056),
             (2000, 8), (700, 12), (300, 512), (257, 516), (99, 1024), (65, 1028), (9, 256), (5, 252)]


def outliers(rng, M, K):
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    return x * np.where(rng.random(K) < 0.02, 30, 1).astype(np.float32)


@pytest.mark.parametrize("M,K", ROW_SIZES)
def test_norm(tb, M, K):
    import torch
    say(f"[norm] {M} x {K}")
    rng = np.random.default_rng(M * 7 + K)
    x, r = outliers(rng, M, K), outliers(rng, M, K)
    w = (1 + 0.3 * rng.normal(0, 1, K)).astype(np.float32)
    for residual in (None, r):
        h, y = ref.add_rms_norm(x, w, 1e-6, residual)
        res = None if residual is None else dev(residual)
        a = tb.bitnet_add_rms_norm(dev(x), dev(w), 1e-6, res)
        assert near(host(a["y"]), y)
        assert ("sum" in a) == (residual is not None)
        if residual is not None:
            assert np.array_equal(host(a["sum"]), h)
        b = tb.bitnet_add_rms_norm(dev(x), dev(w), 1e-6, res, codes=True)
        q, s = ref.quant_rows(host(a["y"]))
        assert np.array_equal(host(b["xq"]), q) and np.array_equal(host(b["x_scale"]), s)
        if K % 128 == 0:
            q2, s2 = tb.bitnet_quant_act(a["y"])
            assert torch.equal(q2, b["xq"]) and torch.equal(s2, b["x_scale"])


@pytest.mark.parametrize("M,K", [(5, 1536), (9, 2052), (3, 12000), (1026, 300)])
def test_norm_in_place_strided_all_outputs(tb, M, K):
    import torch
    say(f"[norm] strided, in place {M} x {K}")
    rng = np.random.default_rng(M + K)
    x, r = outliers(rng, M, K), outliers(rng, M, K)
    w = rng.normal(0, 1, K).astype(np.float32)
    h, y = ref.add_rms_norm(x, w, 1e-5, r)
    wide = torch.full((M, K + 12), float("nan"), device="cuda:0")
    wide[:, 4:4 + K] = dev(x)
    xs, res = wide[:, 4:4 + K], dev(r)
    o = {n: torch.full((M + 1, K), -7, dtype=t, device="cuda:0")
         for n, t in (("y", torch.float32), ("xq", torch.int8))}
    sc = torch.full((M + 1,), -7.0, device="cuda:0")
    tb.bitnet_add_rms_norm_into(M, K, xs, dev(w), 1e-5, res, res, o["y"], o["xq"], sc)
    assert np.array_equal(host(res), h) and near(host(o["y"])[:M], y)
    q, s = ref.quant_rows(host(o["y"])[:M])
    assert np.array_equal(host(o["xq"])[:M], q) and np.array_equal(host(sc)[:M], s)
    assert (host(o["y"])[M:] == -7).all() and (host(o["xq"])[M:] == -7).all() and host(sc)[M] == -7
    xd = dev(x)
    tb.bitnet_add_rms_norm_into(M, K, xd, dev(w), 1e-5, dev(r), xd, o["y"])
    assert np.array_equal(host(xd), h) and near(host(o["y"])[:M], y)


def test_norm_rows_of_zeros_and_extremes(tb):
    say("[norm] zeros, tiny and large rows")
    K = 1536
    x = np.zeros((6, K), np.float32)
    x[1, 3] = 1e-30
    x[2] = 1e18
    x[3] = -1e-22
    x[4, ::2] = 3.0
    w = np.linspace(-2, 2, K).astype(np.float32)
    for eps in (0.0, 1e-6):
        h, y = ref.add_rms_norm(x, w, eps)
        a = host(tb.bitnet_add_rms_norm(dev(x), dev(w), eps)["y"])
        assert near(a, y) and (a[0] == 0).all()
        b = tb.bitnet_add_rms_norm(dev(x), dev(w), eps, codes=True)
        keep = np.abs(a).max(1) > 1e-30   # (127 / max overflows below: outside the contract)
        q, s = ref.quant_rows(a[keep | (np.abs(a).max(1) == 0)])
        assert np.array_equal(host(b["xq"])[keep | (np.abs(a).max(1) == 0)], q)
        assert host(b["x_scale"])[0] == 1.0


@pytest.mark.parametrize("M,K", ROW_SIZES)
def test_gate(tb, M, K):
    import torch
    say(f"[gate] {M} x {K}")
    rng = np.random.default_rng(M * 3 + K)
    g, u = (2 * rng.normal(0, 1, (M, K))).astype(np.float32), outliers(rng, M, K)
    want = ref.silu_mul(g, u)
    a = tb.bitnet_silu_mul(dev(g), dev(u))
    assert near(host(a["y"]), want)
    b = tb.bitnet_silu_mul(dev(g), dev(u), codes=True)
    q, s = ref.quant_rows(host(a["y"]))
    assert np.array_equal(host(b["xq"]), q) and np.array_equal(host(b["x_scale"]), s)
    both = torch.full((M, 2 * K + 8), float("nan"), device="cuda:0")
    both[:, :K], both[:, K + 4:2 * K + 4] = dev(g), dev(u)
    y = torch.full((M + 1, K), -7.0, device="cuda:0")
    xq = torch.full((M + 1, K), -7, dtype=torch.int8, device="cuda:0")
    sc = torch.full((M + 1,), -7.0, device="cuda:0")
    tb.bitnet_silu_mul_into(M, K, both[:, :K], both[:, K + 4:2 * K + 4], y, xq, sc)
    assert torch.equal(y[:M], a["y"]) and torch.equal(xq[:M], b["xq"])
    assert torch.equal(sc[:M], b["x_scale"]) and sc[M] == -7 and (y[M] == -7).all() and (xq[M] == -7).all()
    for t in (dev(g), dev(u)):   # in place
        pair = (t, dev(u)) if torch.equal(t, dev(g)) else (dev(g), t)
        tb.bitnet_silu_mul_into(M, K, *pair, y=t)
        assert torch.equal(t, a["y"])


def test_gate_range(tb):
    """Every size of a gate: far from zero both ways, around it, the smallest."""
    say("[gate] range")
    g = np.concatenate([np.linspace(-800, 800, 4001), np.logspace(-45, 38, 3000),
                        -np.logspace(-45, 38, 3000), [0.0, -0.0], np.linspace(-1e-3, 1e-3, 997)])
    K = 4 * (len(g) // 4)
    g = g[:K].astype(np.float32)[None]
    for up in (1.0, -3.7e-5, 1e-30):
        u = np.full_like(g, up)
        keep = np.abs(ref.silu_mul(g, u)) < 1e38
        got = host(tb.bitnet_silu_mul(dev(np.where(keep, g, 0)), dev(u))["y"])
        assert near(got, ref.silu_mul(np.where(keep, g, 0), u))


# ---- log probabilities -------------------------------------------------------------

def lse_error(R, V):
    t = -(-V // 4096)
    c = min(t, 64, -(-1024 // R))
    return (15 + 4 * -(-t // c) + 2 * math.log(V)) * U


def check_logprobs(tb, x, tokens, top, ld=None):
    import torch
    R, V = x.shape
    if ld:
        wide = torch.full((R, ld), 1e3, device="cuda:0")
        wide[:, :V] = dev(x)
        xd = wide[:, :V]
    else:
        xd = dev(x)
    got = tb.bitnet_token_logprobs(xd, None if tokens is None else dev(tokens), top)
    want = ref.token_logprobs(x, tokens, top)
    e = lse_error(R, V)

    def close(a, b, tol):
        a = a.astype(np.float64)
        inf = np.isneginf(b)
        assert (np.isneginf(a) == inf).all()
        with np.errstate(invalid="ignore"):
            bad = ~inf & ~(np.abs(a - b) <= tol)
        assert not bad.any(), (np.abs(a - b)[bad].max(), e)

    H = want["entropy"]
    close(host(got["entropy"]), H, e + (2 * e + 5 * U) * H)
    if tokens is not None:
        close(host(got["logprobs"]), want["logprobs"], e + U * np.abs(want["logprobs"]))
    if top:
        assert np.array_equal(host(got["top_tokens"]), want["top_tokens"])
        close(host(got["top_logprobs"]), want["top_logprobs"],
              e + U * np.abs(want["top_logprobs"]))
    return got


def some_logits(rng, R, V):
    x = (2.5 * rng.normal(0, 1, (R, V))).astype(np.float32)
    for r in range(R):
        x[r, rng.integers(0, V, 8)] += 6
    x[:, rng.random(V) < 0.1] = -np.inf
    x[:, V // 2] = 1.0
    return x


@pytest.mark.parametrize("R,V,top", [
    (1, 1, 0), (1, 1, 1), (1, 5, 5), (3, 31, 8), (1, 4096, 1), (2, 4097, 9), (16, 151936, 5),
    (1, 151936, 20), (1, 300001, 32), (5, 65536, 32), (17, 9000, 0), (700, 1000, 3),
    (1024, 5000, 2), (1023, 5000, 0), (1500, 12289, 1), (2, 40000, 8),
])
def test_logprobs(tb, R, V, top):
    say(f"[logprobs] {R} x {V} top {top}")
    rng = np.random.default_rng(R + V + top)
    x = some_logits(rng, R, V)
    tokens = rng.integers(0, V, R).astype(np.int32)
    tokens[::5] = x[::5].argmax(1)
    if R > 2:
        tokens[1], tokens[2] = -1, V
    check_logprobs(tb, x, tokens, top, ld=None if R % 2 else V + 5)
    check_logprobs(tb, x[:1], None, top)


def test_logprobs_edges(tb):
    """Rows that mask everything, NaN and infinities, equal logits, one likely
    token, masks of the type's lowest value and of -1e30."""
    say("[logprobs] edges")
    low = np.finfo(np.float32).min
    for V in (7, 5000, 40000):
        x = np.zeros((12, V), np.float32)
        x[0] = -np.inf
        x[1, ::2], x[1, 1::2] = np.nan, np.inf
        x[1, 3] = 2.0
        x[2] = low
        x[3] = low
        x[3, 4] = 5.0
        x[4] = -1e30
        x[5, 2] = 200.0
        x[6, 2] = 15.0
        x[7] = np.linspace(-80, 80, V)
        x[8] = -np.inf
        x[8, V - 1] = -3e38
        x[9] = 1e30
        x[10] = np.linspace(2 ** 24 - 60, 2 ** 24 + 60, V)
        x[11, 1::2] = -0.0
        tokens = np.array([0, 3, 1, 4, 0, 2, 5, V - 1, V - 1, 6, V - 1, 0], np.int32)
        for top in (0, 3, 7):
            check_logprobs(tb, x, tokens, top)


@pytest.mark.parametrize("V,top", [(4096, 32), (4001, 20), (9000, 8), (151936, 32), (70000, 9)])
def test_logprobs_orders(tb, V, top):
    """Rows whose largest lie together: sorted both ways, in one thread's quads, in one
    wave's, in the last chunk, all the same, two values, a few above many equal ones."""
    rng = np.random.default_rng(V + top)
    up = np.arange(V, dtype=np.float32) / V
    one = rng.normal(0, 1, V).astype(np.float32)
    one[4:8] += 20
    one[1028:1032] += 20
    wave = rng.normal(0, 1, V).astype(np.float32)
    wave[256:512] += 20
    last = rng.normal(0, 1, V).astype(np.float32)
    last[-40:] += 20
    few = np.full(V, -3.0, np.float32)
    few[rng.choice(V, top // 2, replace=False)] = 1.0
    x = np.stack([up, up[::-1], one, wave, last, np.full(V, 2.5, np.float32),
                  rng.integers(0, 2, V).astype(np.float32), few])
    check_logprobs(tb, x, rng.integers(0, V, len(x)).astype(np.int32), top)


def test_logprobs_nothing_left_of_a_row_adds_nothing_elsewhere(tb):
    """Outputs that are not asked for are not written, and a row's results do not
    depend on the others'."""
    import torch
    say("[logprobs] single outputs")
    rng = np.random.default_rng(0)
    x = some_logits(rng, 6, 30000)
    tok = rng.integers(0, 30000, 6).astype(np.int32)
    full = tb.bitnet_token_logprobs(dev(x), dev(tok), 4)
    ws = torch.zeros(tb.bitnet_token_logprobs_workspace_bytes(6, 30000, 4), dtype=torch.uint8,
                     device="cuda:0")
    e = torch.full((7,), -7.0, device="cuda:0")
    tb.bitnet_token_logprobs_into(6, 30000, dev(x), None, 0, None, e, None, None, ws)
    assert torch.equal(e[:6], full["entropy"]) and e[6] == -7
    lp = torch.full((7,), -7.0, device="cuda:0")
    tb.bitnet_token_logprobs_into(6, 30000, dev(x), dev(tok), 0, lp, None, None, None, ws)
    assert torch.equal(lp[:6], full["logprobs"]) and lp[6] == -7
    y = x.copy()
    y[[0, 2, 5]] = np.nan
    part = tb.bitnet_token_logprobs(dev(y), dev(tok), 4)
    for n in full:
        assert torch.equal(part[n][[1, 3, 4]], full[n][[1, 3, 4]])
