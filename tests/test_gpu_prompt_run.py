"""The calls around a prompt's projections together, as a decoder uses them: page
map, embedding, norm to 8-bit rows, ternary projections, append, chunk attention,
gated activation, lm_head and log probabilities.  Every call is compared with its
plain definition (fp64) on the inputs it had, with the tolerances of the single
calls' tests; then the same prompts in pieces and token by token, on other streams,
two at once, and captured and replayed, which has to give the same bits."""
import numpy as np
import pytest

from oracle import decode_step, prompt as ref
from tests.test_gpu_decode_step import U, dev, dtype_of, host, rope_tables, say, tb  # noqa: F401
from tests.test_gpu_prompt import LOST, lse_error, near

pytestmark = pytest.mark.gpu

HID, FF, D, KV, G, V, PS, LAYERS, R, TOP = 256, 640, 64, 2, 3, 5000, 8, 2, 3, 5
H = KV * G
PROMPT = (37, 5, 150)


class Decoder:
    """Three requests over a decoder of two layers."""

    def __init__(self, tb, dt, seed=0):
        import torch
        self.tb, self.dt = tb, dt
        rng = np.random.default_rng(seed)
        f = lambda *s: rng.normal(0, 1, s).astype(np.float32)
        w = lambda n, k: (*tb.bitnet_ternarize_pack(dev(f(n, k))), n)
        self.layers = [{"qkv": [w(n * D, HID) for n in (H, KV, KV)], "o": w(HID, H * D),
                        "ff": [w(FF, HID), w(FF, HID)], "down": w(HID, FF),
                        "norm": [dev(1 + 0.2 * f(HID)) for _ in range(2)]} for _ in range(LAYERS)]
        self.table, self.table_scale = tb.bitnet_table_quant(dev(f(V, HID)))
        self.last_norm = dev(1 + 0.2 * f(HID))
        self.cos, self.sin = (dev(a) for a in rope_tables(256, D))
        mp = 32
        self.cache = tb.KvCache.empty(LAYERS, R * mp + 3, KV, PS, D, dtype_of(dt))
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if t is not None:
                t.zero_()
        self.pool, self.state = tb.KvPool.empty(R, mp, R * mp + 3, PS)
        self.ids = [rng.integers(0, V, 200).astype(np.int32) for _ in range(R)]
        torch.cuda.synchronize()

    def tokens(self, done, new):
        """Ids of new tokens behind the first `done`, and the ones that follow them."""
        take = lambda off: dev(np.concatenate([i[d + off:d + off + n]
                                               for i, d, n in zip(self.ids, done, new)]))
        return take(0), take(1), dev(np.array(new, np.int32))

    def run(self, *a, stream=None, **kw):
        with self.tb._on(stream):   # (the projections' outputs are the current stream's)
            return self.forward(*a, stream, **kw)

    def forward(self, ids, following, new, stream, look=lambda *a: None, single=False):
        import torch
        tb = self.tb
        T = ids.shape[0]
        step = tb.bitnet_kv_map(self.pool, T, new, self.state, stream=stream)
        x, delta = tb.bitnet_embed_lookup(ids, self.table, self.table_scale, HID, stream=stream), None
        q8 = lambda r, w: tb.bitnet_ternary_matmul_q8(r["xq"], r["x_scale"], *w, stream=stream)

        def norm(x, delta, weight, codes=True):
            r = tb.bitnet_add_rms_norm(x, weight, 1e-5, delta, codes, stream=stream)
            look("norm", x, delta, weight, r)
            return r.get("sum", x), r

        for l, w in enumerate(self.layers):
            x, r = norm(x, delta, w["norm"][0])
            q, k, v = (q8(r, p) for p in w["qkv"])
            q = tb.bitnet_kv_append(self.cache, l, k, v, step["slots"], step["positions"], self.cos,
                                    self.sin, q, stream=stream)
            if single:
                att = tb.bitnet_paged_attention(self.cache, l, q, self.pool.tables,
                                                step["positions"] + 1, rows=step["rows"],
                                                return_lse=True, stream=stream)
            else:
                att = tb.bitnet_chunk_attention(self.cache, l, q, step["starts"], self.state[:R],
                                                self.pool.tables, return_lse=True, stream=stream)
            look("attend", l, q, step["starts"], *att)
            x, r = norm(x, tb.bitnet_ternary_matmul(att[0], *w["o"], stream=stream), w["norm"][1])
            gate, up = (q8(r, p) for p in w["ff"])
            r = tb.bitnet_silu_mul(gate, up, True, stream=stream)
            look("gate", gate, up, r)
            delta = q8(r, w["down"])
        x, r = norm(x, delta, self.last_norm, False)
        logits = torch.empty(T, V, device="cuda:0")
        for t in range(0, T, 16):
            tb.bitnet_lm_head_into(min(16, T - t), V, HID, r["y"][t:], self.table, self.table_scale,
                                   logits[t:], stream=stream)
        s = tb.bitnet_token_logprobs(logits, following, TOP, stream=stream)
        look("score", logits, following, s)
        return [*step.values(), *att, r["y"], logits, *s.values()]

    def bits(self, out):
        import torch
        torch.cuda.synchronize()
        keep = [*out, self.state, self.pool.tables, self.cache.k, self.cache.v, self.cache.k_scale,
                self.cache.v_scale]
        return [t.contiguous().view(torch.uint8).cpu().numpy().tobytes() for t in keep
                if t is not None]

    def held(self, side, l, r, n):
        """The first n tokens of a request in a layer's cache, fp64 [KV, n, D]."""
        c = self.cache
        t = np.arange(n)
        page, tok = host(self.pool.tables)[r][t // PS], t % PS
        x = host((c.v if side else c.k)[l].double())[page, :, tok]
        sc = c.v_scale if side else c.k_scale
        x = x if sc is None else x * host(sc[l].double())[page, :, tok][..., None]
        return x.transpose(1, 0, 2)


class Check:
    """Every call against its definition; counts what it saw."""

    def __init__(self, d):
        self.d, self.seen = d, {}

    def __call__(self, what, *a):
        self.seen[what] = self.seen.get(what, 0) + 1
        getattr(self, what)(*a)

    def codes(self, r, y):
        """8-bit rows of y, known to half a step of fp32: a code may be the next one
        where y times the scale lies within 127 * 4 u of a border."""
        q, s = host(r["xq"]).astype(np.float64), host(r["x_scale"]).astype(np.float64)
        top = np.abs(y).max(1)
        want = np.where(top > 0, 127 / np.where(top > 0, top, 1), 1)
        assert (np.abs(s - want) <= 4 * U * want).all()
        assert (np.abs(q - y * s[:, None]) <= 0.5 + 127 * 4 * U).all()

    def norm(self, x, delta, weight, r):
        h, y = ref.add_rms_norm(host(x), host(weight), 1e-5, None if delta is None else host(delta))
        if delta is not None:
            assert np.array_equal(host(r["sum"]), h)
        if "y" in r:
            assert near(host(r["y"]), y)
        else:
            self.codes(r, y)

    def gate(self, gate, up, r):
        self.codes(r, ref.silu_mul(host(gate), host(up)))

    def attend(self, l, q, starts, out, lse):
        d = self.d
        q, out, lse = host(q).reshape(-1, H, D), host(out).reshape(-1, H, D), host(lse)
        lens = host(d.state[:R])
        held = [[d.held(side, l, r, n) for r, n in enumerate(lens)] for side in (0, 1)]
        got = ref.chunk_attention(q, host(starts), lens, 256, lambda r, n: held[0][r][:, :n],
                                  lambda r, n: held[1][r][:, :n], D ** -0.5)
        assert set(got) == set(range(len(q)))
        for t, (want, want_lse, smax, mag, n) in got.items():
            lost = n * LOST[d.dt] * max(np.abs(v).max() for v in held[1])
            tol = U * (2 * (D + 16) * smax + 2 * n + 64)[:, None] * mag + lost
            assert (np.abs(out[t] - want) <= tol).all(), (l, t)
            tol = U * ((D + 16) * smax + n + 64) + n * LOST[d.dt] + U * np.abs(want_lse)
            assert (np.abs(lse[t] - want_lse) <= tol).all(), (l, t)

    def score(self, logits, following, s):
        x = host(logits)
        want, e = ref.token_logprobs(x, host(following), TOP), lse_error(*x.shape)
        assert np.array_equal(host(s["top_tokens"]), want["top_tokens"])
        for n in ("logprobs", "top_logprobs"):
            assert (np.abs(host(s[n]) - want[n]) <= e + U * np.abs(want[n])).all(), n
        assert (np.abs(host(s["entropy"]) - want["entropy"]) <=
                e + (2 * e + 5 * U) * want["entropy"]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
def test_prompts_and_steps(tb, dt):  # noqa: F811
    """Whole prompts, then two steps of one and a piece of ragged lengths."""
    say(f"[prompt run] {dt}")
    d = Decoder(tb, dt)
    done = [0] * R
    for new in (PROMPT, (1, 1, 1), (0, 20, 3), (1, 0, 1)):
        look = Check(d)
        d.run(*d.tokens(done, new), look=look)
        assert look.seen == {"norm": 2 * LAYERS + 1, "attend": LAYERS, "gate": LAYERS, "score": 1}
        done = [a + b for a, b in zip(done, new)]
        assert host(d.state)[:R].tolist() == done


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_pieces(tb, dt):  # noqa: F811
    """In pieces, and token by token through the attention of single tokens: the first
    layer's 8-bit rows have the same bits, and every call keeps its tolerance for every
    split.  (The projections' outputs need not: from 17 rows on they take one fp32
    factor a row, w / x rounded, and round its product with the sum, up to 16 rows
    acc * w / x in fp64, rounded once.)"""
    say(f"[prompt run] pieces {dt}")

    class Rows(Check):
        def __init__(self, d, new):
            super().__init__(d)
            self.ends, self.rows = np.cumsum(new)[:-1], None

        def norm(self, x, delta, weight, r):
            super().norm(x, delta, weight, r)
            if self.rows is None:
                bits = np.c_[host(r["xq"]), host(r["x_scale"]).view(np.int8).reshape(-1, 4)]
                self.rows = np.split(bits, self.ends)

    whole, single = Rows(Decoder(tb, dt), PROMPT), Rows(Decoder(tb, dt), PROMPT)
    for look in (whole, single):
        look.d.run(*look.d.tokens([0] * R, PROMPT), look=look, single=look is single)
    pieces, done, rows = Decoder(tb, dt), [0] * R, [[] for _ in range(R)]
    for new in ((30, 1, 64), (0, 4, 1), (7, 0, 85)):
        look = Rows(pieces, new)
        pieces.run(*pieces.tokens(done, new), look=look)
        done = [a + b for a, b in zip(done, new)]
        rows = [a + [b] for a, b in zip(rows, look.rows)]
    for r in range(R):
        assert np.array_equal(whole.rows[r], single.rows[r]), r
        assert np.array_equal(whole.rows[r], np.concatenate(rows[r])), r


PIECES = [(20, 3, 40), (1, 1, 1), (1, 1, 1), (1, 1, 1)]


@pytest.mark.parametrize("dt", ["fp16", "int8"])
def test_on_streams(tb, dt):  # noqa: F811
    """On a stream of its own, and two at once, against the default stream."""
    import torch
    say(f"[prompt run] streams {dt}")
    here, there, beside = (Decoder(tb, dt) for _ in range(3))
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    done = [0] * R
    for new in PIECES:
        args = here.tokens(done, new)
        want = here.bits(here.run(*args))
        a, b = there.run(*args, stream=s), beside.run(*args, stream=t)
        assert there.bits(a) == want and beside.bits(b) == want, new
        done = [a + b for a, b in zip(done, new)]


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_captured(tb, dt):  # noqa: F811
    """A step captured and replayed, the lengths growing by themselves, with eager work
    of two others between the replays."""
    import torch
    say(f"[prompt run] captured {dt}")
    eager, captured, other = (Decoder(tb, dt) for _ in range(3))
    args = eager.tokens([0] * R, PIECES[0])
    for d in (eager, captured, other):
        d.run(*args)
    torch.cuda.synchronize()
    args = [a.clone() for a in eager.tokens(PIECES[0], (1, 1, 2))]
    for d in (eager, captured, other):   # (what runs once before a capture)
        d.run(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.run(*args)
    for turn in range(5):
        want = eager.bits(eager.run(*args))
        graph.replay()
        assert captured.bits(out) == want, turn
        other.run(*args)
        if turn == 1:
            args[0].copy_((args[0] + 17) % V)


def test_two_graphs_with_a_workspace_each(tb):  # noqa: F811
    """Two graphs of the same calls on other inputs, replayed in turn and at once."""
    import torch
    say("[prompt run] two graphs")
    rng = np.random.default_rng(3)
    graphs, outs, wants = [], [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for n in range(2):
        d = Decoder(tb, "bf16", n)
        d.run(*d.tokens([0] * R, PROMPT))
        q = dev(rng.normal(0, 1, (40, H * D)).astype(np.float32))
        starts = dev(np.array([0, 30, 31, 40], np.int32))
        logits = dev(rng.normal(0, 3, (40, 20000)).astype(np.float32))
        ws = torch.zeros(tb.bitnet_token_logprobs_workspace_bytes(40, 20000, 9), dtype=torch.uint8,
                         device="cuda:0")
        cws = torch.empty(tb.bitnet_chunk_attention_workspace_bytes(40, R, H, KV, D, 256),
                          dtype=torch.uint8, device="cuda:0")
        out = [torch.empty(40, H * D, device="cuda:0"), torch.empty(40, device="cuda:0"),
               torch.empty(40, 9, dtype=torch.int32, device="cuda:0"),
               torch.empty(40, 9, device="cuda:0")]

        def run(d=d, q=q, starts=starts, logits=logits, ws=ws, cws=cws, out=out):
            tb.bitnet_chunk_attention_into(d.cache, 1, 40, H, q, starts, d.state[:R], d.pool.tables,
                                           256, 0.125, out[0], cws)
            tb.bitnet_token_logprobs_into(40, 20000, logits, None, 9, None, *out[1:], ws)

        run()
        torch.cuda.synchronize()
        wants.append([host(t).tobytes() for t in out])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
        outs.append(out)
    for turn in range(6):
        for o in outs:
            for t in o:
                t.fill_(-1)
        torch.cuda.synchronize()
        for n in ((0, 1) if turn % 2 else (1, 0)):
            with torch.cuda.stream(streams[n]):
                graphs[n].replay()
        torch.cuda.synchronize()
        assert [[host(t).tobytes() for t in o] for o in outs] == wants, turn


def test_layer_of_the_readme(tb):  # noqa: F811
    """The README's layer around the projections, as it stands there, behind its page map."""
    import os
    import re
    import torch
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S)
                 if "bitnet_chunk_attention" in b]
    assert len(found) == 1
    say("[prompt run] the README's layer")
    rng = np.random.default_rng(4)
    f = lambda *s: dev(rng.normal(0, 1, s).astype(np.float32))
    w = lambda n, k: (*tb.bitnet_ternarize_pack(f(n, k)), n)
    rows, new = 16, rng.integers(0, 40, 16).astype(np.int32)
    T = int(new.sum())
    cache = tb.KvCache.empty(2, 128, KV, PS, D)
    pool, state = tb.KvPool.empty(rows, 8, 128, PS)
    step = tb.bitnet_kv_map(pool, T, dev(new), state)
    cos, sin = (dev(a) for a in rope_tables(64, D))
    ns = {"tb": tb, "cache": cache, "layer": 1, "pool": pool, "state": state, "step": step,
          "cos": cos, "sin": sin, "x": f(T, HID), "delta": f(T, HID), "norm1": f(HID),
          "norm2": f(HID), "wq": w(H * D, HID), "wk": w(KV * D, HID), "wv": w(KV * D, HID),
          "wo": w(HID, H * D), "wg": w(FF, HID), "wu": w(FF, HID), "wd": w(HID, FF),
          "logits": f(T, V), "following": dev(rng.integers(0, V, T).astype(np.int32))}
    x, delta = host(ns["x"]), host(ns["delta"])
    exec(found[0], ns)
    d = Decoder(tb, "bf16")
    d.cache, d.pool, d.state = cache, pool, state
    lens = host(state)[:rows]
    assert (lens == new).all()
    held = [[d.held(s, 1, r, n) for r, n in enumerate(lens)] for s in (0, 1)]
    got = ref.chunk_attention(host(ns["q"]).reshape(-1, H, D), host(step["starts"]), lens, 64,
                              lambda r, n: held[0][r][:, :n], lambda r, n: held[1][r][:, :n], D ** -0.5)
    a = host(ns["a"]).reshape(-1, H, D)
    for t, (want, _, smax, mag, n) in got.items():
        lost = n * LOST["bf16"] * max(np.abs(v).max(initial=0) for v in held[1])
        tol = U * (2 * (D + 16) * smax + 2 * n + 64)[:, None] * mag + lost
        assert (np.abs(a[t] - want) <= tol).all(), t
    back = host(ns["x"]) - host(tb.bitnet_ternary_matmul(ns["a"], *ns["wo"]))
    assert np.allclose(back, x + delta, atol=1e-3)
    Check(d).codes(ns["h"], ref.silu_mul(host(ns["gate"]), host(ns["up"])))
    Check(d).score(ns["logits"], ns["following"], ns["scores"])
    assert torch.isfinite(ns["delta"]).all()
