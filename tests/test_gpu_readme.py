"""The README's decode step, as it stands there, for what its comments allow:
prompts, requests that grow by one token, wait, end and are refused."""
import os
import re

import numpy as np
import pytest

from tests.test_gpu_decode_step import LOST, U, dev, host, rope_tables, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def blocks():
    """The two parts of the example: what is set up once, and a step."""
    with open(os.path.join(ROOT, "README.md")) as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "KvCache.empty" in b]
    assert len(found) == 1
    return found[0].split("\n\n", 1)


def test_decode_step_of_the_readme(tb):  # noqa: F811
    import torch
    setup, step = blocks()
    rng = np.random.default_rng(0)
    D, KV, H, V, rows = 128, 2, 12, 500, 16
    ns = {"tb": tb, "torch": torch, "layer": 3}
    exec(setup, ns)
    assert ns["cache"].head_dim == D and ns["cache"].kv_heads == KV and ns["pool"].rows == rows
    cos, sin = rope_tables(512, D)
    ns.update(cos=dev(cos), sin=dev(sin))
    held = [np.empty((0, 2, KV, D)) for _ in range(rows)]     # a request's keys and values
    lens = np.zeros(rows, np.int64)
    full = 512 * 64
    prompts = rng.integers(1, 300, rows)
    steps = [prompts, np.ones(rows, np.int64), np.ones(rows, np.int64), np.ones(rows, np.int64)]
    steps[1][[1, 7]], steps[1][3] = 0, -1                     # two wait, one ends
    steps[2][3], steps[2][5], steps[2][9] = 40, full + 1, 70  # a prompt, one too long, several tokens
    steps[3][[0, 15]] = -1
    for n, new in enumerate(steps):
        say(f"[readme] step {n}: {new.tolist()}")
        granted = np.where((new > 0) & (lens + new <= full), new, 0)
        lens[new < 0] = 0
        T = int(granted.sum()) + 5                            # and some padding
        of = np.repeat(np.arange(rows), granted)
        pos = np.concatenate([lens[r] + np.arange(c) for r, c in enumerate(granted)])
        q, k, v = (rng.normal(0, 1, (T, c * D)).astype(np.float32) for c in (H, KV, KV))
        # every beam's best token is far above the others, so each follows itself
        logits = np.full((rows, V), -30, np.float32)
        best = rng.integers(0, V, rows)
        logits[np.arange(rows), best] = 10 + rng.random(rows)
        ns.update(T=T, new_lens=dev(new.astype(np.int32)), q=dev(q), k=dev(k), v=dev(v),
                  logits=dev(logits),
                  scores=dev(np.tile(-np.arange(4, dtype=np.float32), rows // 4)))
        exec(step, ns)
        t = len(of)
        c, s = cos[pos][:, None], sin[pos][:, None]

        def turned(x, heads):   # (rounded once to fp32, as the calls say)
            x = x[:t].reshape(t, heads, D).astype(np.float64)
            a, b = x[..., :D // 2], x[..., D // 2:]
            return np.concatenate([a * c - b * s, b * c + a * s], -1).astype(np.float32)

        bf16 = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
        nk, nv = bf16(turned(k, KV)), bf16(v[:t].reshape(t, KV, D))
        for r in range(rows):
            if new[r] < 0:
                held[r] = held[r][:0]
            held[r] = np.concatenate([held[r], np.stack([nk[of == r], nv[of == r]], 1)])
        lens += granted
        assert host(ns["state"])[:rows].tolist() == lens.tolist()
        status = host(ns["step"]["status"])
        assert (status != 0).tolist() == (new > granted).tolist()
        qt = np.zeros((T, H * D), np.float32)
        qt[:t] = turned(q, H).reshape(t, -1)
        out = host(ns["out"])
        assert out.shape == (T, H * D) and (out[t:] == 0).all()
        ks, vs = ([x[:, i].transpose(1, 0, 2) for x in held] for i in (0, 1))
        row_of, seen = np.r_[of, np.zeros(5, int)], np.r_[pos + 1, np.zeros(5, int)]
        check_outputs(out, qt, row_of, seen, ks, vs, D)
        assert host(ns["best"]["tokens"]).tolist() == best.tolist()
        assert host(ns["best"]["parents"]).tolist() == list(range(rows))
        tables = host(ns["pool"].tables)
        for r in range(rows):
            pages = tables[r, :-(-lens[r] // 64)]
            assert (pages >= 0).all() and len(set(pages.tolist())) == len(pages)


def check_outputs(out, q, rows, lens, ks, vs, D):
    """Attention of each token over what its request holds up to it."""
    H, kv = q.shape[1] // D, ks[0].shape[0]
    for t in range(len(rows)):
        n = int(lens[t])
        for h in range(kv if n else 0):
            k, v = ks[rows[t]][h, :n], vs[rows[t]][h, :n]
            x = q[t].reshape(kv, H // kv, D)[h].astype(np.float64)
            s = D ** -0.5 * (x @ k.T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            size = D ** -0.5 * (np.abs(x) @ np.abs(k).T).max(1)
            tol = U * (2 * (D + 16) * size + 2 * n + 64)[:, None] * (p @ np.abs(v))
            tol += n * LOST["bf16"] * np.abs(v).max()
            err = np.abs(out[t].reshape(kv, H // kv, D)[h] - p @ v)
            assert (err <= tol).all(), (t, rows[t], n)
