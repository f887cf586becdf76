"""The calls around a prompt's projections at the ends of what they accept: the
largest sizes and strides, offsets that pass 32 bits, rows of the smallest numbers.
Tolerances are those of tests/test_gpu_prompt.py."""
import numpy as np
import pytest

from oracle import prompt as ref
from tests.test_gpu_decode_step import U, dev, host, say, tb  # noqa: F401
from tests.test_gpu_prompt import LOST, Paged, chunk_case, lse_error, near

pytestmark = pytest.mark.gpu


def normal(gen, *shape):
    import torch
    return torch.randn(shape, generator=gen, device="cuda:0")


@pytest.fixture
def gen():
    import torch
    g = torch.Generator(device="cuda:0")
    g.manual_seed(5)
    yield g
    torch.cuda.empty_cache()


# ---- chunk attention --------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "int8"])
def test_chunk_far_pages(tb, dtype):  # noqa: F811
    """A cache of more than 2^32 bytes: pages behind that, layers further apart."""
    import torch
    say(f"[prompt range] far pages {dtype}")
    rng = np.random.default_rng(1)
    lens, new = np.array([300, 77]), np.array([40, 77])
    pg = Paged(tb, rng, dtype, lens, 2, 128, 16, layers=2, layer=1)
    P = (1 << 32) // (16 * 2 * 128 * pg.kd.element_size()) + 1000
    far = rng.permutation(np.r_[P - 500:P])[:pg.P]

    def spread(t):
        if t is None:
            return None
        big = torch.zeros((2, P, *t.shape[2:]), dtype=t.dtype, device="cuda:0")
        big[:, dev(far)] = t
        return big

    big = [spread(t) for t in (pg.kd, pg.vd, pg.ksd, pg.vsd)]
    cache = tb.KvCache(*big)
    assert big[0][1].numel() * big[0].element_size() > 1 << 32
    q = rng.normal(0, 1, (117, 12, 128)).astype(np.float32)
    starts = np.array([0, 40, 117])
    tables = np.where(pg.tables >= 0, far[np.maximum(pg.tables, 0)], -1).astype(np.int32)
    out, lse = tb.bitnet_chunk_attention(cache, 1, dev(q.reshape(117, -1)), dev(starts.astype(np.int32)),
                                         dev(lens.astype(np.int32)), dev(tables), return_lse=True)
    rows = pg.check(q, starts, lens, pg.mp * 16, 128 ** -0.5, host(out).reshape(q.shape), host(lse))
    assert len(rows) == 117


def test_chunk_of_many_rows(tb, gen):  # noqa: F811
    """Rows, outputs and strides that pass 2^32 bytes, 4096 requests."""
    import torch
    R, H, KV, D, PS = 4096, 128, 8, 128, 32
    say("[prompt range] chunk attention of 69,632 rows of 128 heads")
    rng = np.random.default_rng(2)
    more = rng.integers(-17, 18, R // 2)
    new = 17 + rng.permutation(np.r_[more, -more])
    T = int(new.sum())
    lens = new + rng.integers(0, 31, R)
    assert T == 17 * R and lens.max() <= 3 * PS
    pages = torch.randint(0, 50, (R, 3), generator=gen, device="cuda:0", dtype=torch.int32)
    k, v = (normal(gen, 1, 50, KV, PS, D).to(torch.bfloat16) for _ in range(2))
    cache = tb.KvCache(k, v)
    starts = np.r_[0, np.cumsum(new)]
    stride = H * D + 64
    q = torch.empty(T, stride, device="cuda:0")
    for part in q.split(4096):
        part.copy_(normal(gen, *part.shape))
    qd = q[:, :H * D]
    out, lse = tb.bitnet_chunk_attention(cache, 0, qd, dev(starts.astype(np.int32)),
                                         dev(lens.astype(np.int32)), pages, return_lse=True)
    assert q.numel() * 4 > 1 << 32 and out.numel() * 4 > 1 << 32
    kh, vh, ph = host(k[0].double()), host(v[0].double()), host(pages)
    for r in np.r_[0, rng.integers(0, R, 60), R - 1]:
        n = int(lens[r])
        t = np.arange(n)
        rows = [x[ph[r][t // PS], :, t % PS].transpose(1, 0, 2) for x in (kh, vh)]
        part = slice(int(starts[r]), int(starts[r + 1]))
        qr = host(qd[part]).reshape(-1, H, D)
        got, e = host(out[part]).reshape(-1, H, D), host(lse[part])
        want = ref.chunk_attention(qr, [0, len(qr)], [n], 96, lambda _, m: rows[0][:, :m],
                                   lambda _, m: rows[1][:, :m], D ** -0.5)
        for i, (o, w, smax, mag, m) in want.items():
            tol = U * (2 * (D + 16) * smax + 2 * m + 64)[:, None] * mag
            assert (np.abs(got[i] - o) <= tol).all(), (r, i)
            assert (np.abs(e[i] - w) <= U * ((D + 16) * smax + m + 64 + np.abs(w))).all()


@pytest.mark.parametrize("max_len", [1, 5, 64, 65])
def test_chunk_small_max_len(tb, max_len):  # noqa: F811
    """Lengths beyond max_len count as that: more rows than tokens that can be seen."""
    chunk_case(tb, max_len, "fp16", [3, 90, 1], [200, 0, 64], 2, 6, 128, 16, max_len=max_len)


@pytest.mark.parametrize("PS", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("dtype", ["fp16", "int8"])
def test_chunk_small_pages(tb, dtype, PS):  # noqa: F811
    chunk_case(tb, PS, dtype, [70, 1, 0, 9], [300, 90, 5, 0], 2, 5, 64 if PS > 2 else 256, PS,
               heads_first=PS % 4 == 0)


def test_chunk_far_strides(tb):  # noqa: F811
    """Tokens of a page 2^26 elements apart: 16 of them are not at 32-bit offsets."""
    import torch
    say("[prompt range] far strides")
    rng = np.random.default_rng(4)
    lens, new = np.array([60, 33]), np.array([20, 33])
    pg = Paged(tb, rng, "bf16", lens, 1, 64, 16, spare_pages=0)
    far, P = 1 << 26, pg.P
    store = torch.zeros(16 * far + P * 64, dtype=torch.bfloat16, device="cuda:0")
    apart = lambda: torch.as_strided(store, (1, P, 1, 16, 64), (1 << 31, 64, 64, far, 1))
    caches = []
    for t in (pg.kd, pg.vd):
        a = apart()
        a.copy_(t)
        caches.append(a)
        if len(caches) == 1:
            store = torch.zeros_like(store)
    cache = tb.KvCache(*caches)
    q = rng.normal(0, 1, (53, 4, 64)).astype(np.float32)
    starts = np.array([0, 20, 53])
    out, lse = tb.bitnet_chunk_attention(cache, 0, dev(q.reshape(53, -1)), dev(starts.astype(np.int32)),
                                         dev(lens.astype(np.int32)), dev(pg.tables.astype(np.int32)),
                                         return_lse=True)
    rows = pg.check(q, starts, lens, pg.mp * 16, 64 ** -0.5, host(out).reshape(q.shape), host(lse))
    assert len(rows) == 53


# ---- norm and gated activation ----------------------------------------------------

def sample(rng, M):
    return np.unique(np.r_[0, 1, M - 2, M - 1, rng.integers(0, M, 40)])


def quantized(y, q, s):
    wq, ws = ref.quant_rows(y)
    return np.array_equal(q, wq) and np.array_equal(s, ws)


@pytest.mark.parametrize("M,K,stride", [((1 << 23) - 1, 4, 4), (300_000, 8960, 8960),
                                        (6, 1536, (1 << 31) - 4), (66_000, 32768, 32768)])
def test_norm_largest(tb, gen, M, K, stride):  # noqa: F811
    import torch
    say(f"[prompt range] norm {M} x {K}, rows {stride} apart")
    rng = np.random.default_rng(M)
    buf = torch.empty((M - 1) * stride + K, device="cuda:0")
    x = torch.as_strided(buf, (M, K), (stride, 1))
    if stride == K:
        for part in x.split(max(1, (1 << 27) // K)):
            part.copy_(normal(gen, *part.shape))
    else:
        x.copy_(normal(gen, M, K))
    w = normal(gen, K)
    a = tb.bitnet_add_rms_norm(x, w, 1e-6)["y"]
    b = tb.bitnet_add_rms_norm(x, w, 1e-6, codes=True)
    rows = sample(rng, M)
    at = dev(rows)
    _, y = ref.add_rms_norm(host(x[at]), host(w), 1e-6)
    got = host(a[at])
    assert near(got, y)
    assert quantized(got, host(b["xq"][at]), host(b["x_scale"][at]))


@pytest.mark.parametrize("M,K,stride", [((1 << 23) - 1, 8, 16), (150_000, 8960, 17920),
                                        (6, 12000, (1 << 31) - 4)])
def test_gate_largest(tb, gen, M, K, stride):  # noqa: F811
    """Gate and up as halves of one tensor, whose rows lie far apart."""
    import torch
    say(f"[prompt range] gate {M} x {K}, rows {stride} apart")
    rng = np.random.default_rng(M)
    buf = torch.empty((M - 1) * stride + 2 * K, device="cuda:0")
    both = torch.as_strided(buf, (M, 2 * K), (stride, 1))
    for part in both.split(max(1, (1 << 27) // K)):
        part.copy_(2 * normal(gen, *part.shape))
    g, u = both[:, :K], both[:, K:]
    a = tb.bitnet_silu_mul(g, u)["y"]
    b = tb.bitnet_silu_mul(g, u, codes=True)
    at = dev(sample(rng, M))
    got = host(a[at])
    assert near(got, ref.silu_mul(host(g[at]), host(u[at])))
    assert quantized(got, host(b["xq"][at]), host(b["x_scale"][at]))


@pytest.mark.parametrize("K", [128, 8960, 12032])
def test_rows_of_the_smallest_numbers(tb, K):  # noqa: F811
    """Where 127 / max overflows, scale and codes are those of the quantization of the
    call's fp32 row all the same."""
    import torch
    say(f"[prompt range] smallest numbers {K}")
    rng = np.random.default_rng(K)
    mag = np.float32(2.0) ** rng.integers(-149, -118, (40, 1))
    x = (rng.normal(0, 1, (40, K)) * mag).astype(np.float32)
    x[:, ::5] = 0
    x[3], x[4] = 0, 1e-45
    one = np.ones(K, np.float32)
    for call in (lambda c: tb.bitnet_add_rms_norm(dev(x), dev(one), 1.0, codes=c),
                 lambda c: tb.bitnet_silu_mul(dev(80 * np.abs(np.sign(x))), dev(x / 64), codes=c)):
        a, b = call(False)["y"], call(True)
        q, s = tb.bitnet_quant_act(a)
        assert torch.isinf(s).any() and torch.equal(s, b["x_scale"]) and torch.equal(q, b["xq"])


# ---- log probabilities --------------------------------------------------------------

def test_logprobs_most_rows(tb, gen):  # noqa: F811
    """65,535 rows, logits that pass 2^32 elements."""
    import torch
    R, V, ld, top = 65535, 5000, 70001, 6
    say("[prompt range] log probabilities of 65,535 rows")
    rng = np.random.default_rng(7)
    x = torch.empty((R - 1) * ld + V, device="cuda:0")
    x = torch.as_strided(x, (R, V), (ld, 1))
    for part in x.split(8192):
        part.copy_(3 * normal(gen, *part.shape))
    tokens = dev(rng.integers(-1, V + 1, R).astype(np.int32))
    got = tb.bitnet_token_logprobs(x, tokens, top)
    at = dev(sample(rng, R))
    want, e = ref.token_logprobs(host(x[at]), host(tokens[at]), top), lse_error(R, V)
    assert np.array_equal(host(got["top_tokens"][at]), want["top_tokens"])
    for n in ("logprobs", "top_logprobs"):
        assert (np.abs(host(got[n][at]) - want[n]) <= e + U * np.abs(want[n])).all(), n
    assert (np.abs(host(got["entropy"][at]) - want["entropy"]) <=
            e + (2 * e + 5 * U) * want["entropy"]).all()
    # every row: the largest is the largest, and its log probability is plausible
    for r0 in range(0, R, 8192):
        part = slice(r0, min(R, r0 + 8192))
        v, i = x[part].double().max(1)
        lse = torch.logsumexp(x[part].double(), 1)
        assert torch.equal(got["top_tokens"][part, 0].long(), i)
        assert ((got["top_logprobs"][part, 0].double() - (v - lse)).abs() <=
                e + U * (v - lse).abs() + 1e-12).all()


@pytest.mark.parametrize("top", [0, 3, 32])
def test_logprobs_largest_vocabulary(tb, gen, top):  # noqa: F811
    """2^30 - 1 logits of a row."""
    import torch
    V = (1 << 30) - 1
    say(f"[prompt range] 2^30 - 1 logits, top {top}")
    x = torch.empty(1, V, device="cuda:0")
    for part in x[0].split(1 << 27):
        part.copy_(normal(gen, part.numel()))
    best = [V - 1, 5, V // 2, 0, V - 2] + [1000 + 7_000_001 * i for i in range(30)]
    x[0, torch.tensor(best, device="cuda:0")] = torch.arange(60, 25, -1, device="cuda:0") / 4.0
    S = W = 0.0
    for part in x[0].split(1 << 26):
        d = part.double()
        e = d.exp()
        S += float(e.sum())
        W += float((e * d).sum())
    lse = np.log(S)
    got = tb.bitnet_token_logprobs(x, dev(np.array([V // 2], np.int32)), top)
    e, H = lse_error(1, V), lse - W / S
    say(f"  entropy off by {abs(float(got['entropy']) - H) / U:.0f} u of {(e + (2 * e + 5 * U) * H) / U:.0f}")
    assert abs(float(got["logprobs"]) - (58 / 4 - lse)) <= e + U * abs(58 / 4 - lse)
    assert abs(float(got["entropy"]) - H) <= e + (2 * e + 5 * U) * H
    if top:
        assert host(got["top_tokens"])[0].tolist() == best[:top]
        w = np.arange(60, 60 - top, -1) / 4 - lse
        assert (np.abs(host(got["top_logprobs"])[0] - w) <= e + U * np.abs(w)).all()


# ---- chunk attention: scales and magnitudes -----------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.25, 1e-30, -3.0])
def test_chunk_of_any_scale(tb, dtype, scale):  # noqa: F811
    chunk_case(tb, 31, dtype, [70, 1, 33], [300, 64, 0], 2, 3, 128, 16, scale=scale)


@pytest.mark.parametrize("q2,k2,v2", [(-100, 100, 0), (118, -118, 0), (100, -100, -110), (0, 0, 120),
                                      (58, 58, 0), (50, 50, 100)])
@pytest.mark.parametrize("D", [64, 256])
def test_chunk_of_any_magnitude(tb, D, q2, k2, v2):  # noqa: F811
    """bf16 caches near the ends of fp32: queries 2^-100 to 2^118, scores up to 2^122."""
    import torch
    from tests.test_gpu_prompt import run_chunk
    say(f"[prompt range] chunk of q 2^{q2}, k 2^{k2}, v 2^{v2}")
    rng = np.random.default_rng(6)
    new, old = np.array([70, 1, 40]), np.array([0, 32, 560])
    pg = Paged(tb, rng, "bf16", new + old, 2, D, 16)
    for t, f in ((pg.kd, k2), (pg.vd, v2)):
        t.copy_(torch.ldexp(t.float(), torch.tensor(f, device="cuda:0")).bfloat16())
    pg.make(tb)
    q = rng.normal(0, 1, (111, 6, D)).astype(np.float32) * np.float32(2.0 ** q2)
    run_chunk(tb, pg, q, np.r_[0, np.cumsum(new)], new + old, 6, scale=0.125)


@pytest.mark.parametrize("k2,v2,uneven", [(0, 0, 20), (-90, 0, 0), (60, 0, 0), (0, -90, 0), (0, 90, 0),
                                          (0, -60, 30), (0, 0, 0)])
def test_chunk_of_any_scales_of_rows(tb, k2, v2, uneven):  # noqa: F811
    """8-bit caches: scales far from one, value scales up to 2^`uneven` apart, zeros."""
    from tests.test_gpu_prompt import run_chunk
    say(f"[prompt range] chunk of row scales 2^{k2}, 2^{v2}, {uneven} apart")
    rng = np.random.default_rng(8)
    new, old = np.array([70, 1, 40]), np.array([0, 90, 300])
    pg = Paged(tb, rng, "int8", new + old, 2, 128, 16)
    pg.ksd *= 2.0 ** k2
    pg.vsd *= dev((2.0 ** v2 * 2.0 ** -rng.integers(0, uneven + 1, pg.vsd.shape)).astype(np.float32))
    pg.vsd[0, ::3] = 0
    pg.ks, pg.vs = host(pg.ksd), host(pg.vsd)
    pg.make(tb)
    q = (rng.normal(0, 1, (111, 12, 128)) * 2.0 ** -k2).astype(np.float32)
    run_chunk(tb, pg, q, np.r_[0, np.cumsum(new)], new + old, 12)


def test_chunk_scores_of_thousands(tb):  # noqa: F811
    """Scores of thousands, rising and falling along the length: the base moves often."""
    import torch
    from tests.test_gpu_prompt import run_chunk
    rng = np.random.default_rng(9)
    for dtype in ("bf16", "fp16", "int8"):
        for order in (1, -1):
            say(f"[prompt range] rising scores {dtype} {order}")
            pg = Paged(tb, rng, dtype, [700], 1, 128, 32)
            ramp = torch.linspace(*((0.2, 4) if order > 0 else (4, 0.2)), 736, device="cuda:0")
            for j in range(-(-700 // 32)):
                page = int(pg.tables[0, j])
                row = ramp[32 * j:32 * j + 32]
                if dtype == "int8":
                    pg.ksd[0, page, 0] = row * 0.03
                else:
                    pg.kd[0, page, 0] *= row[:, None].to(pg.kd.dtype)
            if dtype == "int8":
                pg.ks = host(pg.ksd)
            pg.make(tb)
            q = (40 * rng.normal(0, 1, (90, 6, 128))).astype(np.float32)
            run_chunk(tb, pg, q, [0, 90], [700], 6, scale=0.5)
