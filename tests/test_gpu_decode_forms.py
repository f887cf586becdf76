"""The allocating forms of the decode-step calls on a stream of their own, and
captured into a graph and replayed, against the same calls on the default stream."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import dev, host, rope_tables, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu

L, R, W, KV, H, D, PS, V = 2, 8, 4, 2, 6, 128, 16, 9000


class Step:
    """One step's inputs, and the five calls on them."""

    def __init__(self, tb, dtype):
        import torch
        rng = np.random.default_rng(1)
        self.tb = tb
        f = lambda *s: dev(rng.normal(0, 1, s).astype(np.float32))
        self.cache = tb.KvCache.empty(L, 64, KV, PS, D, dtype)
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if t is not None:
                t.zero_()
        self.pool, self.state = tb.KvPool.empty(R, 6, 64, PS)
        self.cos, self.sin = (dev(a) for a in rope_tables(100, D))
        self.T = R * 5
        self.new = torch.full((R,), 5, dtype=torch.int32, device="cuda:0")
        self.q, self.k, self.v = f(self.T, H * D), f(self.T, KV * D), f(self.T, KV * D)
        self.logits, self.scores = f(R, V), f(R)
        self.fin = dev((np.arange(R) % 3 == 0).astype(np.int32))
        torch.cuda.synchronize()

    def run(self, stream=None):
        tb, out = self.tb, []
        step = tb.bitnet_kv_map(self.pool, self.T, self.new, self.state, stream=stream)
        out += list(step.values())
        for layer in range(L):
            q = tb.bitnet_kv_append(self.cache, layer, self.k, self.v, step["slots"],
                                    step["positions"], self.cos, self.sin, self.q, stream=stream)
            out += [q, *tb.bitnet_paged_attention(self.cache, layer, q, self.pool.tables,
                                                  self.lens(step, stream), rows=step["rows"],
                                                  return_lse=True, stream=stream)]
        best = tb.bitnet_beam_select(self.logits, self.scores, W, self.fin, 7, stream=stream)
        tables = tb.bitnet_beam_reorder(self.cache, self.pool.tables, self.state[:R],
                                        best["parents"], W, stream=stream)
        return out + list(best.values()) + [tables]

    def lens(self, step, stream):
        import torch
        with torch.cuda.stream(stream):
            return step["positions"] + 1

    def bits(self, out):
        import torch
        torch.cuda.synchronize()
        keep = [*out, self.state, self.pool.tables, self.pool.owned, self.pool.free_pages,
                self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale]
        return [t.contiguous().view(torch.uint8).cpu().numpy().tobytes() for t in keep
                if t is not None]


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_on_a_stream(tb, dt):  # noqa: F811
    import torch
    say(f"[forms] stream {dt}")
    dtype = torch.int8 if dt == "int8" else torch.bfloat16
    here, there = Step(tb, dtype), Step(tb, dtype)
    s = torch.cuda.Stream()
    for turn in range(3):
        assert here.bits(here.run()) == there.bits(there.run(s)), turn


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_captured(tb, dt):  # noqa: F811
    import torch
    say(f"[forms] captured {dt}")
    dtype = torch.int8 if dt == "int8" else torch.bfloat16
    eager, captured, other = (Step(tb, dtype) for _ in range(3))
    for s in (eager, captured, other):
        first = s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.run()
    for turn in range(4):
        want = eager.bits(eager.run())
        graph.replay()
        assert captured.bits(out) == want, turn
        other.run()
    assert len(first) == len(out)
