"""Plain definitions of the calls around a prompt's projections, for the tests.

numpy and Python loops, fp64 where floating point, one statement per rule of
the header; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

from . import decode_step


def request_rows(T, starts, lens, max_len):
    """[(request, row, tokens the row attends to)] of the rows that are a request's."""
    out, at = [], 0
    edge = []
    for s in starts:
        at = max(at, int(s))
        edge.append(min(at, T))
    for r, (a, b) in enumerate(zip(edge, edge[1:])):
        total = min(max(int(lens[r]), 0), max_len)
        out += [(r, t, max(total - (b - a) + (t - a) + 1, 0)) for t in range(a, b)]
    return out


def chunk_attention(q, starts, lens, max_len, keys, values, scale):
    """q fp32 [T, H, D]; keys(r, n), values(r, n): the first n tokens of request r
    that are there, fp64 [kv heads, <= n, D] -> dict of row -> (out [H, D], lse [H],
    magnitudes as decode_step.attention gives them, tokens)."""
    return {t: (*decode_step.attention(q[t], keys(r, n), values(r, n), scale), n)
            for r, t, n in request_rows(len(q), starts, lens, max_len)}


def quant_rows(y):
    """fp32 [M, K] -> int8 codes and scales: 127 / max, half to even."""
    top = np.abs(y).max(1)
    with np.errstate(divide="ignore"):
        s = np.where(top == 0, np.float32(1), np.float32(127) / top).astype(np.float32)
    return np.clip(np.rint((y * s[:, None]).astype(np.float32)), -127, 127).astype(np.int8), s


def add_rms_norm(x, weight, eps, residual=None):
    """-> h fp32 and y fp64 of it."""
    h = x if residual is None else (x + residual).astype(np.float32)
    d = h.astype(np.float64)
    under = (d * d).sum(1, keepdims=True) / d.shape[1] + float(np.float32(eps))
    with np.errstate(divide="ignore", invalid="ignore"):
        y = d * weight.astype(np.float64) / np.sqrt(under)
    return h, np.where(under > 0, y, 0.0)


def silu_mul(gate, up):
    g = gate.astype(np.float64)
    with np.errstate(over="ignore"):
        return g * up.astype(np.float64) / (1.0 + np.exp(-g))


def token_logprobs(logits, tokens=None, top=0):
    """-> dict of fp64 logprobs, entropy, top_logprobs and int32 top_tokens."""
    R, V = logits.shape
    out = {"entropy": np.zeros(R), "logprobs": np.zeros(R),
           "top_tokens": np.zeros((R, top), np.int32), "top_logprobs": np.zeros((R, top))}
    for r in range(R):
        x = logits[r].astype(np.float64)
        x = np.where(x < np.inf, x, -np.inf)
        m, lse = x.max(), 0.0
        if m > -np.inf:
            e = np.exp(x - m)
            lse = m + np.log(e.sum())
            p = e / e.sum()
            out["entropy"][r] = -(p[p > 0] * np.log(p[p > 0])).sum()
        best = np.lexsort((np.arange(V), -x))[:top]
        out["top_tokens"][r], out["top_logprobs"][r] = best, x[best] - lse
        if tokens is not None and 0 <= tokens[r] < V:
            out["logprobs"][r] = x[tokens[r]] - lse
    return out
