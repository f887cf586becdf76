"""Plain definitions of the cache and beam-search calls, for the tests.

numpy and Python loops, fp64 where floating point, one statement per rule of
the header; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def kv_map(page_size, pages, T, new_lens, state, tables, owned, free_pages):
    """The page map of one step; returns a dict of new arrays."""
    B, mp = tables.shape
    tables, owned, free = tables.copy(), owned.copy(), free_pages.copy()
    ps = page_size
    lens = [int(min(max(x, 0), mp * ps)) for x in state[:B]]
    held = [int(min(max(x, 0), mp)) for x in state[B:2 * B]]
    height = int(min(max(state[2 * B], 0), pages))
    for r in range(B):
        if new_lens[r] < 0:
            for i in range(held[r]):
                if height < pages:
                    free[height] = owned[r, i]
                    height += 1
            lens[r] = held[r] = 0
    status = np.zeros(B, np.int32)
    slots, positions, rows = (np.full(T, -1, np.int32) for _ in range(3))
    starts = np.zeros(B + 1, np.int32)
    want_pages = want_tokens = used = 0
    t = 0
    for r in range(B):
        starts[r] = t
        n = max(int(new_lens[r]), 0)
        have = -(-lens[r] // ps)
        need = -(-(lens[r] + n) // ps) - have
        if lens[r] + n > mp * ps or held[r] + need > mp:
            status[r] = 1
            continue
        want_pages += need
        want_tokens += n
        if need and want_pages > height:
            status[r] = 2
        elif n and want_tokens > T:
            status[r] = 3
        if status[r]:
            continue
        for i in range(need):
            page = free[height - 1 - used]
            tables[r, have + i] = page
            owned[r, held[r] + i] = page
            used += 1
        for p in range(lens[r], lens[r] + n):
            page = int(tables[r, p // ps])
            slots[t] = page * ps + p % ps if 0 <= page < pages else -1
            positions[t], rows[t] = p, r
            t += 1
        lens[r] += n
        held[r] += need
    starts[B] = t
    out = np.array(lens + held + [height - used], np.int32)
    return {"state": out, "starts": starts, "slots": slots, "positions": positions, "rows": rows,
            "status": status, "tables": tables, "owned": owned, "free": free}


def rotate(x, cos, sin):
    """x fp32 [T, heads, D] turned by cos, sin [T, D/2]: fp64, rounded to fp32."""
    h = x.shape[-1] // 2
    a, b = x[..., :h].astype(np.float64), x[..., h:].astype(np.float64)
    c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64)
    return np.concatenate([a * c - b * s, b * c + a * s], -1).astype(np.float32)


def quant_rows(x):
    """fp32 [..., D] -> int8 codes and fp32 scales [...] of the 8-bit cache."""
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x / s[..., None]).astype(np.float32))
    q = np.where(s[..., None] == 0, 0, np.clip(q, -127, 127))
    return q.astype(np.int8), s


def attention(q, k, v, scale):
    """q [H, D], k and v [heads, n, D] (fp64 values) -> out [H, D], lse [H] and
    the two magnitudes that error bounds need: max_j scale * sum |q k_j| and
    sum_j p_j |v_j|."""
    H, D = q.shape
    kv, n = k.shape[:2]
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    smax, mag = np.zeros(H), np.zeros((H, D))
    for h in range(H if n else 0):
        kh, vh = k[h // (H // kv)], v[h // (H // kv)]
        s = scale * (kh @ q[h].astype(np.float64))
        m = s.max()
        p = np.exp(s - m)
        lse[h] = m + np.log(p.sum())
        p /= p.sum()
        out[h], mag[h] = p @ vh, p @ np.abs(vh)
        smax[h] = (abs(scale) * (np.abs(kh) @ np.abs(q[h].astype(np.float64)))).max()
    return out, lse, smax, mag


def beam_select(logits, scores, W, finished=None, eos=-1):
    """Candidates sorted by (score, beam, logit, token); returns a dict with
    fp64 scores, plus the smallest gap between scores of different beams."""
    R, V = logits.shape
    out = {"scores": np.zeros(R), "tokens": np.zeros(R, np.int32), "parents": np.zeros(R, np.int32),
           "finished": np.zeros(R, np.int32)}
    gap = np.inf
    for g in range(0, R, W):
        cand = []
        for r in range(g, g + W):
            base = float(scores[r]) if scores[r] < np.inf else -np.inf
            if finished is not None and finished[r]:
                cand.append((-base, r, -1.0, eos))
                cand += [(np.inf, r, 0.0, t) for t in range(min(W + 1, V)) if t != eos]
                continue
            x = logits[r].astype(np.float64)
            x = np.where(x < np.inf, x, -np.inf)
            m = x.max()
            lse = m + np.log(np.exp(x - m).sum()) if m > -np.inf else 0.0
            best = np.lexsort((np.arange(V), -x))[:W]
            cand += [(-(base + (x[t] - lse)), r, -x[t], int(t)) for t in best]
        cand.sort()
        for a, b in zip(cand[:W], cand[1:W + 1]):
            if a[1] != b[1] and a[0] < np.inf and a[0] != b[0]:
                gap = min(gap, b[0] - a[0])
        for j, (s, r, _, t) in enumerate(cand[:W]):
            out["scores"][g + j], out["tokens"][g + j], out["parents"][g + j] = -s, t, r
            if finished is not None:
                out["finished"][g + j] = int(bool(finished[r]) or t == eos)
    out["gap"] = gap
    return out


def beam_reorder(k, v, k_scale, v_scale, W, parents, lens, tables):
    """Caches [layers, pages, heads, page, D] (copied) and tables of the new
    beams."""
    arrays = [None if a is None else a.copy() for a in (k, v, k_scale, v_scale)]
    pages, ps = k.shape[1], k.shape[3]
    R, mp = tables.shape
    out = tables.copy()
    for g in range(0, R, W):
        n = min(max(int(lens[g]), 0), mp * ps)
        last, tail = n // ps, n % ps
        par = [int(p) if g <= p < g + W else g + j for j, p in enumerate(parents[g:g + W])]
        spare = [r for r in range(g, g + W) if r not in par]
        kept = set()
        for j, p in enumerate(par):
            out[g + j, :last] = tables[p, :last]
            if not tail:
                continue
            giver = p
            if p in kept:
                giver = spare.pop(0)
                src, dst = int(tables[p, last]), int(tables[giver, last])
                if 0 <= src < pages and 0 <= dst < pages:
                    for a in arrays:
                        if a is not None:
                            a[:, dst, :, :tail] = a[:, src, :, :tail]
            kept.add(p)
            out[g + j, last] = tables[giver, last]
    return (*arrays, out)
