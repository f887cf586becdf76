"""The cache and beam-search calls together, as a decode loop uses them: page
map, embedding, ternary projections, append, attention, lm_head, selection and
reordering, for a prompt and the steps after it.  Every call is compared with
its plain definition (oracle/decode_step.py, fp64) on the inputs it had; then
the same loop is captured into a graph, and run on other streams, and has to
give the same bits.  Tolerances are those of the single calls' tests."""
import numpy as np
import pytest

from oracle import decode_step as ref
from tests.test_gpu_decode_step import LOST, U, dev, dtype_of, host, rope_tables, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu

HID, D, KV, G, V, PS, LAYERS = 256, 64, 2, 2, 500, 8, 2
H = KV * G


class Loop:
    """B groups of W beams over a two-layer decoder; every buffer is allocated
    here, so that a step only launches."""

    def __init__(self, tb, dt, B, W, prompt, seed=0):
        import torch
        self.tb, self.B, self.W, self.R, self.dt = tb, B, W, B * W, dt
        rng = np.random.default_rng(seed)
        R, T = self.R, sum(prompt) * W
        f32 = dict(dtype=torch.float32, device="cuda:0")
        i32 = dict(dtype=torch.int32, device="cuda:0")
        w = lambda n, k: tb.bitnet_ternarize_pack(dev(rng.normal(0, 1, (n, k)).astype(np.float32)))
        self.weights = [{"q": w(H * D, HID), "k": w(KV * D, HID), "v": w(KV * D, HID),
                         "o": w(HID, H * D)} for _ in range(LAYERS)]
        self.table, self.table_scale = tb.bitnet_table_quant(
            dev(rng.normal(0, 1, (V, HID)).astype(np.float32)))
        self.cos, self.sin = (dev(a) for a in rope_tables(64, D))
        mp = 8
        self.cache = tb.KvCache.empty(LAYERS, R * mp + 3, KV, PS, D, dtype_of(dt))
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if t is not None:
                t.zero_()
        self.pool, self.state = tb.KvPool.empty(R, mp, R * mp + 3, PS)
        n = max(T, R)
        self.slots, self.pos, self.rows = (torch.empty(n, **i32) for _ in range(3))
        self.starts, self.status = torch.empty(R + 1, **i32), torch.empty(R, **i32)
        self.x, self.o = torch.empty(n, HID, **f32), torch.empty(n, HID, **f32)
        self.q, self.qr, self.att = (torch.empty(n, H * D, **f32) for _ in range(3))
        self.k, self.v = (torch.empty(n, KV * D, **f32) for _ in range(2))
        self.lse = torch.empty(n, H, **f32)
        self.logits = torch.empty(R, V, **f32)
        self.scores = torch.full((R,), -np.inf, **f32)
        self.scores[::W] = 0.0
        self.fin, self.parents = torch.zeros(R, **i32), torch.empty(R, **i32)
        self.tokens = torch.empty(R, **i32)
        self.tables = torch.empty(R, mp, **i32)
        self.ones = torch.ones(R, **i32)
        self.max_len = mp * PS
        zeros = lambda b: torch.zeros(b, dtype=torch.uint8, device="cuda:0")
        self.mm_ws = zeros(tb.bitnet_matmul_workspace_bytes(n, HID))
        self.at_ws = zeros(tb.bitnet_paged_attention_workspace_bytes(n, H, KV, D, self.max_len))
        self.se_ws = zeros(tb.bitnet_beam_select_workspace_bytes(B, W, V))
        ids = [rng.integers(0, V, p).tolist() for p in prompt]
        self.prompt_ids = dev(np.array([t for p in ids for _ in range(W) for t in p], np.int32))
        self.prompt_lens = dev(np.repeat(np.array(prompt, np.int32), W))
        self.prompt_last = dev(np.cumsum(np.repeat(prompt, W)) - 1)
        torch.cuda.synchronize()

    def forward(self, T, ids, lens, stream, look):
        """T tokens: pages, layers; x[:T] at the end."""
        import torch
        tb = self.tb
        look("map", T)
        tb.bitnet_embed_lookup_into(ids, T, self.table, self.table_scale, V, HID, self.x, stream)
        for l, w in enumerate(self.weights):
            for n, out, N in (("q", self.q, H * D), ("k", self.k, KV * D), ("v", self.v, KV * D)):
                tb.bitnet_ternary_matmul_into(T, N, HID, self.x, *w[n], out, self.mm_ws,
                                              stream=stream)
            tb.bitnet_kv_append_into(self.cache, l, T, H, self.k[:T], self.v[:T], self.slots[:T],
                                     self.pos[:T], self.cos, self.sin, self.q[:T], self.qr,
                                     stream)
            look("append", T, l)
            tb.bitnet_paged_attention_into(self.cache, l, T, H, self.qr[:T], self.pool.tables, lens,
                                           self.max_len, D ** -0.5, self.att, self.at_ws,
                                           self.rows[:T], self.lse, stream)
            look("attend", T, l, lens)
            tb.bitnet_ternary_matmul_into(T, HID, H * D, self.att, *w["o"], self.o, self.mm_ws,
                                          stream=stream)
            torch.add(self.x[:T], self.o[:T], out=self.x[:T])

    def choose(self, x, stream, look):
        import torch
        tb = self.tb
        tb.bitnet_lm_head_into(self.R, V, HID, x, self.table, self.table_scale, self.logits,
                               stream=stream)
        look("before select")
        tb.bitnet_beam_select_into(self.B, self.W, V, self.logits, self.scores, self.fin, 2,
                                   self.scores, self.tokens, self.parents, self.fin, self.se_ws,
                                   stream)
        look("select")
        tb.bitnet_beam_reorder_into(self.cache, self.B, self.W, self.parents, self.state,
                                    self.pool.tables, self.tables, stream)
        look("reorder")
        torch.add(self.tables, 0, out=self.pool.tables)

    def map(self, T, new, stream):
        self.tb.bitnet_kv_map_into(self.pool, T, new, self.state, self.state, self.starts,
                                   self.slots, self.pos, self.rows, self.status, stream)

    def prompt(self, stream=None, look=lambda *a: None):
        import torch
        T = self.prompt_ids.numel()
        look("before map", self.prompt_lens)
        self.map(T, self.prompt_lens, stream)
        self.forward(T, self.prompt_ids, self.pos[:T] + 1, stream, look)
        self.choose(self.x[self.prompt_last].contiguous(), stream, look)

    def step(self, stream=None, look=lambda *a: None):
        look("before map", self.ones)
        self.map(self.R, self.ones, stream)
        self.forward(self.R, self.tokens, self.state[:self.R], stream, look)
        self.choose(self.x, stream, look)

    def outputs(self):
        import torch
        torch.cuda.synchronize()
        return [host(t).tobytes() for t in (self.tokens, self.parents, self.scores, self.fin,
                                            self.logits, self.state, self.pool.tables)]


class Check:
    """Follows the loop with the plain definitions."""

    def __init__(self, loop):
        self.s = loop

    def bits(self):
        import torch
        c = self.s.cache
        view = lambda t: None if t is None else host(
            t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()]))
        return [view(t) for t in (c.k, c.v, c.k_scale, c.v_scale)]

    def values(self, l, side, page, tok):
        c = self.s.cache
        x = host((c.v if side else c.k)[l].double())[page, :, tok]
        sc = c.v_scale if side else c.k_scale
        return x if sc is None else x * host(sc[l].double())[page, :, tok][..., None]

    def __call__(self, what, *a):
        s = self.s
        getattr(self, what.replace(" ", "_"))(s, *a)

    def before_map(self, s, new):
        self.new = host(new)
        self.was = [host(t) for t in (s.state, s.pool.tables, s.pool.owned, s.pool.free_pages)]

    def map(self, s, T):
        want = ref.kv_map(PS, s.pool.pages, T, self.new, *self.was)
        got = dict(state=s.state, starts=s.starts, slots=s.slots[:T], positions=s.pos[:T],
                   rows=s.rows[:T], status=s.status, tables=s.pool.tables, owned=s.pool.owned,
                   free=s.pool.free_pages)
        for n, w in want.items():
            assert np.array_equal(host(got[n]), w), n
        assert (want["status"] == 0).all()
        self.before = self.bits()

    def append(self, s, T, l):
        import torch
        cos, sin = host(s.cos), host(s.sin)
        pos, slots = host(s.pos[:T]), host(s.slots[:T])
        turn = lambda t: ref.rotate(host(t[:T]).reshape(T, -1, D), cos[pos], sin[pos])
        assert host(s.qr[:T]).tobytes() == turn(s.q).tobytes()
        want = self.before
        for side, x in enumerate((turn(s.k), host(s.v[:T]).reshape(T, KV, D))):
            if s.dt == "int8":
                x, scale = ref.quant_rows(x)
                want[2 + side][l, slots // PS, :, slots % PS] = scale.view(np.int32)
            else:
                x = torch.from_numpy(x).to(dtype_of(s.dt)).view(torch.int16).numpy()
            want[side][l, slots // PS, :, slots % PS] = x
        for got, w in zip(self.bits(), want):
            assert w is None or np.array_equal(got, w)

    def attend(self, s, T, l, lens):
        q, out, lse = (host(t[:T]) for t in (s.qr, s.att, s.lse))
        tables, rows, lens = host(s.pool.tables), host(s.rows[:T]), host(lens)
        for t in range(T):
            n = lens[t]
            j = np.arange(n)
            page = tables[rows[t], j // PS]
            k, v = (self.values(l, side, page, j % PS).transpose(1, 0, 2) for side in (0, 1))
            o, e, smax, mag = ref.attention(q[t].reshape(H, D), k, v, D ** -0.5)
            tol = U * (2 * (D + 16) * smax[:, None] + 2 * n + 64) * mag
            tol += n * LOST[s.dt] * np.abs(v).max()
            assert (np.abs(out[t].reshape(H, D) - o) <= tol).all(), (l, t)
            assert (np.abs(lse[t] - e) <= U * ((D + 16) * smax + n + 64 + 2 * np.abs(e))).all()

    def before_select(self, s):
        self.chosen = ref.beam_select(host(s.logits), host(s.scores), s.W, host(s.fin), 2)
        assert self.chosen["gap"] > 2 * U * (24 + 2)

    def select(self, s):
        for n, t in (("tokens", s.tokens), ("parents", s.parents), ("finished", s.fin)):
            assert np.array_equal(host(t), self.chosen[n]), n
        exact, got = self.chosen["scores"], host(s.scores).astype(np.float64)
        assert (np.abs(got - exact) <= U * (np.abs(exact) + 64)).all()
        self.before = self.bits()

    def reorder(self, s):
        *want, tables = ref.beam_reorder(*self.before, s.W, host(s.parents), host(s.state),
                                         host(s.pool.tables))
        assert np.array_equal(host(s.tables), tables)
        for got, w in zip(self.bits(), want):
            assert w is None or np.array_equal(got, w)


@pytest.mark.parametrize("dt,B,W,prompt", [("bf16", 2, 3, [13, 8]), ("fp16", 1, 8, [5]),
                                           ("int8", 3, 2, [16, 1, 7]), ("int8", 4, 1, [30, 9, 2, 12])])
def test_prompt_and_steps(tb, dt, B, W, prompt):  # noqa: F811
    say(f"[run] {dt} B={B} W={W} prompt={prompt}")
    loop = Loop(tb, dt, B, W, prompt)
    check = Check(loop)
    loop.prompt(look=check)
    for step in range(10):
        say(f"[run] step {step}")
        loop.step(look=check)


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_captured_steps_replay(tb, dt):  # noqa: F811
    """One captured step, replayed with another loop's eager steps between the
    replays, against the eager loop."""
    import torch
    say(f"[run] captured {dt}")
    eager, captured, other = (Loop(tb, dt, 2, 4, [9, 20]) for _ in range(3))
    for loop in (eager, captured, other):
        loop.prompt()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    assert captured.outputs() == eager.outputs()   # a capture runs nothing
    for step in range(8):
        eager.step()
        graph.replay()
        other.step()
        assert captured.outputs() == eager.outputs() == other.outputs(), step


def test_streams(tb):  # noqa: F811
    """Two loops queued in turn on two streams of their own, each with its own
    workspaces, against the same loop on the default stream."""
    import torch
    say("[run] two streams")
    loops = [Loop(tb, "bf16", 2, 4, [9, 20]) for _ in range(3)]
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for loop, s in zip(loops, streams):
        with torch.cuda.stream(s):
            loop.prompt(s)
    for step in range(6):
        for loop, s in zip(loops, streams):
            with torch.cuda.stream(s):
                loop.step(s)
        if step % 3 == 2:
            want = loops[0].outputs()
            assert loops[1].outputs() == want and loops[2].outputs() == want, step


# ---- sizes that the single calls' tests leave out --------------------------------

@pytest.mark.parametrize("dt", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("T,kv,gq,dim,longest", [(65, 2, 6, 128, 700), (300, 1, 2, 64, 90),
                                                 (1024, 1, 1, 64, 40), (1025, 1, 1, 64, 40),
                                                 (1500, 2, 2, 64, 70), (70, 4, 33, 64, 130),
                                                 (65, 1, 3, 256, 300)])
def test_attention_of_many_rows(tb, dt, T, kv, gq, dim, longest):  # noqa: F811
    """More rows than a wave has lanes, than the split of the length looks at,
    more heads than one product's columns; every fifth row empty, all rows over
    four requests' pages."""
    from tests.test_gpu_decode_step import attend_inputs
    say(f"[run] attention {dt} T={T} kv={kv} G={gq} D={dim}")
    ps = 16
    base = [longest, longest // 2 + 1, 17, 1]
    caches, tables, _, ks, vs = attend_inputs(T, base, longest // ps + 2, kv, gq, dim, ps, dt)
    rng = np.random.default_rng(T)
    rows = rng.integers(0, 4, T).astype(np.int32)
    lens = np.array([rng.integers(1, base[r] + 1) for r in rows], np.int32)
    lens[::5] = 0
    q = rng.normal(0, 1, (T, kv * gq * dim)).astype(np.float32)
    out, lse = tb.bitnet_paged_attention(tb.KvCache(*caches), 1, dev(q), dev(tables), dev(lens),
                                         rows=dev(rows), return_lse=True)
    out, lse = host(out), host(lse)
    heads = kv * gq
    for t in range(T):
        k, v = ks[rows[t]][:, :lens[t]], vs[rows[t]][:, :lens[t]]
        o, e, smax, mag = ref.attention(q[t].reshape(heads, dim), k, v, dim ** -0.5)
        tol = U * (2 * (dim + 16) * smax[:, None] + 2 * lens[t] + 64) * mag
        tol += lens[t] * LOST[dt] * np.abs(v).max(initial=0.0)
        err = np.abs(out[t].reshape(heads, dim) - o)
        assert (err <= tol).all(), (t, float((err - tol).max()))
        if lens[t] == 0:
            assert (lse[t] == -np.inf).all()
        else:
            assert (np.abs(lse[t] - e) <= U * ((dim + 16) * smax + lens[t] + 64
                                               + 2 * np.abs(e))).all(), t


@pytest.mark.parametrize("kv,gq,dim,lens", [
    (1, 1, 64, [2048]), (1, 1, 64, [2049]), (1, 3, 128, [4096, 4097]), (1, 1, 64, [32767]),
    (1, 9, 64, [40000]), (1, 1, 128, [131072]), (2, 2, 64, [33000, 0, 2100, 64, 31]),
    (1, 2, 256, [9000, 8200]), (1, 1, 64, [70000, 60000] + [1500] * 40),
])
def test_attention_of_many_parts(tb, kv, gq, dim, lens):  # noqa: F811
    """Rows cut into 16, 17, 32 and more parts, up to the most there can be:
    groups of parts that are full, hold one part or a few."""
    from tests.test_gpu_decode_step import attend_inputs, check_attention
    say(f"[run] attention in parts kv={kv} G={gq} D={dim} {lens[:4]}")
    ps = 64
    caches, tables, q, ks, vs = attend_inputs(dim, lens, -(-max(lens) // ps), kv, gq, dim, ps,
                                              "bf16")
    cache = tb.KvCache(*caches)
    first = None
    for _ in range(3):
        out, lse = tb.bitnet_paged_attention(cache, 1, dev(q), dev(tables),
                                             dev(np.array(lens, np.int32)), return_lse=True)
        out, lse = host(out), host(lse)
        assert first is None or first == out.tobytes() + lse.tobytes()
        first = out.tobytes() + lse.tobytes()
    check_attention(out, lse, q, ks, vs, dim ** -0.5, dim, LOST["bf16"])


@pytest.mark.parametrize("dt,pages", [("bf16", 150000), ("int8", 280000)])
def test_cache_past_32_bits(tb, dt, pages):  # noqa: F811
    """Pages whose offsets pass 2^31 elements and 2^32 bytes, in the first layer
    and (past twice that) in the second: append, attention, reordering."""
    import torch
    kv, dim, ps, n = 2, 128, 64, 100
    say(f"[run] {dt} cache of {pages} pages")
    cache = tb.KvCache.empty(2, pages, kv, ps, dim, dtype_of(dt))
    assert cache.k[0].numel() > 2 ** 31 and cache.k[0].nbytes > 2 ** 32
    tables = np.array([[pages - 1, pages - 2], [pages - 3, 5]], np.int32)
    rng = np.random.default_rng(1)
    x = [rng.normal(0, 1, (n, kv, dim)).astype(np.float32) for _ in range(4)]
    j = np.arange(n)
    for layer in range(2):
        for r in range(2):
            slots = dev((tables[r][j // ps] * ps + j % ps).astype(np.int32))
            tb.bitnet_kv_append(cache, layer, dev(x[2 * r].reshape(n, -1)),
                                dev(x[2 * r + 1].reshape(n, -1)), slots)
    def stored(a):
        if dt == "int8":
            c, s = ref.quant_rows(a)
            return c.astype(np.float64) * s[..., None]
        return host(torch.from_numpy(a).to(dtype_of(dt)).double())
    vals = [stored(a).transpose(1, 0, 2) for a in x]
    q = rng.normal(0, 1, (2, kv * 3 * dim)).astype(np.float32)

    def check(tables, who):
        for layer in range(2):
            out = host(tb.bitnet_paged_attention(cache, layer, dev(q), tables,
                                                 dev(np.full(2, n, np.int32))))
            for r in range(2):
                o, _, smax, mag = ref.attention(q[r].reshape(-1, dim), vals[2 * who[r]],
                                                vals[2 * who[r] + 1], dim ** -0.5)
                tol = U * (2 * (dim + 16) * smax[:, None] + 2 * n + 64) * mag
                tol += n * LOST[dt] * np.abs(vals[2 * who[r] + 1]).max()
                assert (np.abs(out[r].reshape(-1, dim) - o) <= tol).all(), (layer, r)

    check(dev(tables), [0, 1])
    new = tb.bitnet_beam_reorder(cache, dev(tables), dev(np.full(2, n, np.int32)),
                                 dev(np.array([1, 1], np.int32)), 2)
    assert host(new).tolist() == [[pages - 3, 5], [pages - 3, pages - 2]]
    check(new, [1, 1])


def test_workspaces_are_not_passed(tb):  # noqa: F811
    """Workspaces of exactly the stated size between guards, whose counters are
    zero after every call."""
    import torch
    from tests.test_gpu_decode_step import attend_inputs
    say("[run] workspace guards")
    guard = 4096

    def guarded(size):
        t = torch.zeros(size + 2 * guard, dtype=torch.uint8, device="cuda:0")
        t[:guard] = 0xA5
        t[guard + size:] = 0xA5
        return t, t[guard:guard + size]

    def intact(t, size, header):
        return ((t[:guard] == 0xA5).all() & (t[guard + size:] == 0xA5).all()
                & (t[guard:guard + header] == 0).all()).item()

    for lens, kv, gq, dim, ps in [([32000], 2, 6, 128, 64), ([5000, 3, 900], 1, 17, 64, 16),
                                  ([3000] * 20, 2, 1, 256, 64)]:
        mp = -(-max(lens) // ps)
        caches, tables, q, _, _ = attend_inputs(3, lens, mp, kv, gq, dim, ps, "bf16")
        size = tb.bitnet_paged_attention_workspace_bytes(len(lens), kv * gq, kv, dim, mp * ps)
        t, ws = guarded(size)
        out = torch.empty(len(lens), kv * gq * dim, device="cuda:0")
        for _ in range(2):
            tb.bitnet_paged_attention_into(tb.KvCache(*caches), 1, len(lens), kv * gq, dev(q),
                                           dev(tables), dev(np.array(lens, np.int32)), mp * ps, 0.1,
                                           out, ws)
            assert intact(t, size, min(size, 16384)), (lens, kv, gq)
    for B, W, vocab in [(1, 1, 151936), (32, 8, 30000), (1, 32, 50000), (4096, 1, 40), (2, 5, 9)]:
        size = tb.bitnet_beam_select_workspace_bytes(B, W, vocab)
        t, ws = guarded(size)
        x = torch.randn(B * W, vocab, device="cuda:0")
        s = torch.zeros(B * W, device="cuda:0")
        o = [torch.empty(B * W, device="cuda:0")] + [
            torch.empty(B * W, dtype=torch.int32, device="cuda:0") for _ in range(2)]
        for _ in range(2):
            tb.bitnet_beam_select_into(B, W, vocab, x, s, None, 0, *o, None, ws)
            assert intact(t, size, 32768), (B, W, vocab)
