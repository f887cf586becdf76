"""Operators around a prompt's projections: cases, plain forms and exact values.

Four entry points are described here, each by the cases of a table: attention
of the new tokens of several requests over their pages (``chunk``), the
residual addition with the root-mean-square norm (``norm``), the gated
activation (``gate``), both with fp32 rows or 8-bit rows and scales as their
output, and the log probabilities of given tokens with the entropy and the
likeliest alternatives (``score``).  With ``own`` false, ``run`` computes them
with elementary torch operations; with ``own`` true it makes the calls of the
library.  Head counts (12 query heads on 2 key/value heads of 128 channels),
widths (1536 and 8960), the vocabulary of 151,936 and the lengths 256 and 1800
(30 s and 4 min of audio) are those of the decoder this library serves; the
other sizes are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}


def listed():
    return [
        # the last four tokens of a prompt of one stream, or four guessed ones:
        # the smallest call, where latency counts
        {"name": "chunk_tail", "op": "chunk", "requests": 1, "new_lo": 4, "new_hi": 4, "old_lo": 253,
         "old_hi": 253, "kv": 2, "group": 6, "dim": 128, "page": 64, "type": "bf16",
         "heads_first": True},
        # a 4-minute prompt in one piece
        {"name": "chunk_prompt", "op": "chunk", "requests": 1, "new_lo": 1800, "new_hi": 1800,
         "old_lo": 0, "old_hi": 0, "kv": 2, "group": 6, "dim": 128, "page": 16, "type": "fp16",
         "heads_first": False},
        # a server's step: 16 streams at different places of their prompts, 8-bit pages
        {"name": "chunk_batch", "op": "chunk", "requests": 16, "new_lo": 1, "new_hi": 256,
         "old_lo": 0, "old_hi": 1800, "kv": 2, "group": 6, "dim": 128, "page": 16, "type": "int8",
         "heads_first": True},
        # a piece of a prompt far into the decoder's 32k context
        {"name": "chunk_long", "op": "chunk", "requests": 1, "new_lo": 450, "new_hi": 450,
         "old_lo": 32317, "old_hi": 32317, "kv": 2, "group": 6, "dim": 128, "page": 64,
         "type": "bf16", "heads_first": True},
        # a decode step of 16 streams: fp32 rows for the projections of up to 16 rows
        {"name": "norm_step", "op": "norm", "rows": 16, "width": 1536, "codes": False},
        # a 4-minute prompt: 8-bit rows for the projections of more rows
        {"name": "norm_prompt", "op": "norm", "rows": 1800, "width": 1536, "codes": True},
        # 16 such prompts, the norm before the table: fp32 rows
        {"name": "norm_batch", "op": "norm", "rows": 28800, "width": 1536, "codes": False},
        # between gate, up and down of a decode step of 16 streams
        {"name": "gate_step", "op": "gate", "rows": 16, "width": 8960, "codes": False},
        # the same of a 4-minute prompt, 8-bit rows
        {"name": "gate_prompt", "op": "gate", "rows": 1800, "width": 8960, "codes": True},
        # one stream's token with 20 alternatives
        {"name": "score_one", "op": "score", "rows": 1, "vocab": 151936, "top": 20},
        # 16 streams, 5 alternatives each
        {"name": "score_step", "op": "score", "rows": 16, "vocab": 151936, "top": 5},
        # every token of a 4-minute prompt, no alternatives
        {"name": "score_prompt", "op": "score", "rows": 1800, "vocab": 151936, "top": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "norm", "gate", "score"])
    if op == "chunk":
        kv = rng.choice([1, 2, 2, 3, 4])
        group = rng.choice([1, 2, 4, 5, 6, 7, 8, 12, 16])
        requests = _log(rng, 1, 32)
        new = _log(rng, 1, 2000)
        # scores of all padded rows and tokens, and the padded tokens themselves
        while requests * kv * group * new > 1 << 16:
            new = max(1, new // 2)
            requests = max(1, requests // 2)
        cap = min(32768, (1 << 26) // (requests * kv * max(group * new, 64)))
        old = _log(rng, 1, max(1, cap - new))
        return {"op": op, "requests": requests, "new_lo": rng.randint(0, new), "new_hi": new,
                "old_lo": rng.randint(0, old), "old_hi": old, "kv": kv, "group": group,
                "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([8, 16, 32, 64, 128]),
                "type": rng.choice(["bf16", "fp16", "int8"]), "heads_first": rng.random() < 0.5}
    if op in ("norm", "gate"):
        width = 4 * _log(rng, 16, 2240)
        rows = _log(rng, 1, min(28800, (1 << 24) // width))
        return {"op": op, "rows": rows, "width": width, "codes": rng.random() < 0.5}
    top = rng.choice([0, 0, 1, 2, 5, 8, 20, 32])
    return {"op": op, "rows": _log(rng, 1, 1800 if top == 0 else 64),
            "vocab": _log(rng, 1000, 151936), "top": top}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _spread(g, lo, hi, n):
    """n whole numbers evenly from hi down to lo, in any order, int32."""
    v = hi - torch.arange(n, device="cuda") * (hi - lo) // max(n - 1, 1)
    return v[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _activations(g, rows, channels):
    """N(0, 1) rows whose channels have 1% outliers of twenty times the size."""
    x = torch.randn(rows, channels, generator=g, device="cuda")
    return x * torch.where(torch.rand(channels, generator=g, device="cuda") < 0.01, 20.0, 1.0)


def _pages(g, pages, kv, page, dim, dtype, heads_first):
    """A cache tensor of one layer, indexed [layer, page, head, token, channel];
    in memory heads before tokens, or tokens before heads."""
    shape = (1, pages, kv, page, dim) if heads_first else (1, pages, page, kv, dim)
    if dtype is torch.int8:
        t = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    else:
        t = torch.randn(shape, generator=g, device="cuda").to(dtype)
    return t if heads_first else t.transpose(2, 3)


def _scales(g, pages, kv, page):
    """Scales of 8-bit rows: a row's largest magnitude, 2 to 5, over 127."""
    u = torch.rand(1, pages, kv, page, generator=g, device="cuda")
    return (2.0 + 3.0 * u) / 127.0


def prepare(case, seed):
    st = {"case": case}
    globals()["_prepare_" + case["op"]](case, _gen(seed), st)
    if own:
        globals()["_plan_" + case["op"]](case, st)
    return st


def _prepare_chunk(case, g, st):
    R, kv, D, ps = case["requests"], case["kv"], case["dim"], case["page"]
    H = kv * case["group"]
    dtype = DTYPES[case["type"]]
    new = _spread(g, case["new_lo"], case["new_hi"], R)
    lens = new + _spread(g, case["old_lo"], case["old_hi"], R)
    starts = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    starts[1:] = new.cumsum(0)
    mp = (case["new_hi"] + case["old_hi"] + ps - 1) // ps
    P = R * mp
    tables = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(R, mp)
    col = torch.arange(mp, device="cuda", dtype=torch.int32)
    tables[col[None, :] >= ((lens + ps - 1) // ps)[:, None]] = -1
    st["k"] = _pages(g, P, kv, ps, D, dtype, case["heads_first"])
    st["v"] = _pages(g, P, kv, ps, D, dtype, case["heads_first"])
    if dtype is torch.int8:
        st["ks"], st["vs"] = _scales(g, P, kv, ps), _scales(g, P, kv, ps)
    T = int(starts[-1])                    # a program knows how many tokens it feeds
    st["q"] = torch.randn(T, H * D, generator=g, device="cuda")
    st.update(R=R, T=T, H=H, kv=kv, D=D, ps=ps, mp=mp, lens=lens, starts=starts, tables=tables,
              most=case["new_hi"], scale=1.0 / math.sqrt(D),
              max_len=case["new_hi"] + case["old_hi"])


def _prepare_norm(case, g, st):
    M, K = case["rows"], case["width"]
    # the residual stream has outlier channels, a projection's output less so
    st["residual"] = _activations(g, M, K)
    st["x"] = torch.randn(M, K, generator=g, device="cuda")
    st["weight"] = 1.0 + 0.3 * torch.randn(K, generator=g, device="cuda")
    st.update(M=M, K=K, eps=1e-6, codes=case["codes"])


def _prepare_gate(case, g, st):
    M, K = case["rows"], case["width"]
    # gate and up come from one grouped projection, into buffers of their own
    st["gate"] = 2.0 * torch.randn(M, K, generator=g, device="cuda")
    st["up"] = _activations(g, M, K)
    st.update(M=M, K=K, codes=case["codes"])


def _prepare_score(case, g, st):
    R, V = case["rows"], case["vocab"]
    # logits with a few strong tokens; a tenth of the vocabulary is masked out
    x = torch.randn(R, V, generator=g, device="cuda")
    x *= 2.5
    strong = torch.randint(0, V, (R, 8), generator=g, device="cuda")
    x.scatter_add_(1, strong, 6.0 + 2.0 * torch.randn(R, 8, generator=g, device="cuda"))
    out = torch.rand(V, generator=g, device="cuda") < 0.1
    x.masked_fill_(out, -math.inf)
    # a given token is one of the strong ones, or any that is not masked
    token = torch.where(torch.rand(R, generator=g, device="cuda") < 0.7, strong[:, 0],
                        torch.randint(0, V, (R,), generator=g, device="cuda"))
    st["logits"] = x
    st["tokens"] = torch.where(out[token], (~out).long().argmax(), token).to(torch.int32)
    st.update(R=R, V=V, top=case["top"])


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _binding():
    from ternary_weight_decoder_amd import binding
    return binding


def _plan_chunk(case, st):
    tb = _binding()
    st["cache"] = tb.KvCache(st["k"], st["v"], st.get("ks"), st.get("vs"))
    st["out"] = torch.empty_like(st["q"])
    st["ws"] = torch.zeros(
        tb.bitnet_chunk_attention_workspace_bytes(st["T"], st["R"], st["H"], st["kv"], st["D"],
                                                  st["max_len"]),
        dtype=torch.uint8, device="cuda")


def _plan_rows(st, like):
    if st["codes"]:
        st["xq"] = torch.empty(like.shape, dtype=torch.int8, device="cuda")
        st["xs"] = torch.empty(st["M"], device="cuda")
    else:
        st["y"] = torch.empty_like(like)


def _plan_norm(case, st):
    st["sum"] = torch.empty_like(st["x"])
    _plan_rows(st, st["x"])


def _plan_gate(case, st):
    _plan_rows(st, st["up"])


def _plan_score(case, st):
    tb = _binding()
    R, top = st["R"], st["top"]
    st["out"] = {"logprobs": torch.empty(R, device="cuda"),
                 "entropy": torch.empty(R, device="cuda")}
    st["out"]["top_tokens"] = (torch.empty(R, top, dtype=torch.int32, device="cuda")
                               if top else None)
    st["out"]["top_logprobs"] = torch.empty(R, top, device="cuda") if top else None
    st["ws"] = torch.zeros(tb.bitnet_token_logprobs_workspace_bytes(R, st["V"], top),
                           dtype=torch.uint8, device="cuda")


def _own_chunk(st):
    _binding().bitnet_chunk_attention_into(st["cache"], 0, st["T"], st["H"], st["q"], st["starts"],
                                           st["lens"], st["tables"], st["max_len"], st["scale"],
                                           st["out"], st["ws"])
    return st["out"]


def _rows_out(st):
    """fp32 rows, or the values that 8-bit rows stand for with their scales."""
    if st["codes"]:
        return {"x": torch.div(st["xq"], st["xs"][:, None]), "scale": st["xs"]}
    return {"y": st["y"]}


def _own_norm(st):
    _binding().bitnet_add_rms_norm_into(st["M"], st["K"], st["x"], st["weight"], st["eps"],
                                        st["residual"], st["sum"], st.get("y"), st.get("xq"),
                                        st.get("xs"))
    return dict(_rows_out(st), sum=st["sum"])


def _own_gate(st):
    _binding().bitnet_silu_mul_into(st["M"], st["K"], st["gate"], st["up"], st.get("y"),
                                    st.get("xq"), st.get("xs"))
    return _rows_out(st)


def _own_score(st):
    out = st["out"]
    _binding().bitnet_token_logprobs_into(st["R"], st["V"], st["logits"], st["tokens"], st["top"],
                                          out["logprobs"], out["entropy"], out["top_tokens"],
                                          out["top_logprobs"], st["ws"])
    return out


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _gather(st, name, scales):
    """A cache's tokens in request order, fp32 [requests, heads, tokens, channels]."""
    R, mp, ps = st["R"], st["mp"], st["ps"]
    page = st["tables"].long().clamp(min=0)
    x = st[name][0][page]                                  # [R, mp, kv, ps, D]
    x = x.transpose(1, 2).reshape(R, st["kv"], mp * ps, st["D"]).float()
    if scales in st:
        sc = st[scales][0][page].transpose(1, 2).reshape(R, st["kv"], mp * ps, 1)
        x = x * sc
    return x


def _plain_chunk(st):
    R, T, H, kv, D, most = st["R"], st["T"], st["H"], st["kv"], st["D"], st["most"]
    G, n = H // kv, st["mp"] * st["ps"]
    starts = st["starts"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(most, device="cuda")
    live = i < new[:, None]                                # [R, most]
    row = torch.where(live, starts[:-1, None] + i, 0)
    sees = st["lens"][:, None] - new[:, None] + i + 1      # tokens that a row attends to
    q = st["q"].view(T, kv, G, D)[row]                     # [R, most, kv, G, D]
    q = q.permute(0, 2, 3, 1, 4).reshape(R, kv, G * most, D)
    s = torch.matmul(q, _gather(st, "k", "ks").transpose(-1, -2)) * st["scale"]
    seen = torch.arange(n, device="cuda") < sees[:, :, None]
    s = s.view(R, kv, G, most, n).masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    o = torch.matmul(p.view(R, kv, G * most, n), _gather(st, "v", "vs"))
    o = o.view(R, kv, G, most, D) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(R * most, H * D)
    out = torch.empty(T + 1, H * D, device="cuda")
    return out.index_copy_(0, torch.where(live, row, T).view(-1), o)[:T]


def _plain_rows(y, codes):
    """fp32 rows, or their 8-bit codes' values: rounding of values next to a
    border is decided by the fp32 row, so that is made in 64 bits and rounded
    once."""
    if not codes:
        return {"y": y}
    top = y.abs().amax(-1)
    # (a number over an fp32 tensor is a reciprocal and a product, rounded twice)
    scale = torch.where(top == 0, 1.0, (127.0 / top.double()).float())
    q = torch.round(y * scale[:, None]).clamp(-127, 127).to(torch.int8)
    return {"x": torch.div(q, scale[:, None]), "scale": scale}


def _plain_norm(st):
    h = st["x"] + st["residual"]
    d = h.double()
    r = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + st["eps"])
    y = (d * r * st["weight"].double()).float()
    return dict(_plain_rows(y, st["codes"]), sum=h)


def _plain_gate(st):
    d = st["gate"].double()
    y = (d / (1.0 + torch.exp(-d)) * st["up"].double()).float()
    return _plain_rows(y, st["codes"])


def _plain_score(st):
    R, V, top = st["R"], st["V"], st["top"]
    x = st["logits"]
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    d = x - m
    e = torch.exp(d)
    s = e.sum(-1)
    t = torch.where(e > 0, e * d, 0.0).sum(-1)
    log_s = torch.log(s)
    out = {"logprobs": d.gather(1, st["tokens"].long()[:, None])[:, 0] - log_s,
           "entropy": log_s - t / s, "top_tokens": None, "top_logprobs": None}
    if top:
        # larger logits first, then lower tokens
        i = (x + 0.0).view(torch.int32).long()
        i = torch.where(i < 0, i ^ 0x7fffffff, i)
        tok = (i * (1 << 32) + (0xffffffff - torch.arange(V, device="cuda"))).topk(top).indices
        out.update(top_tokens=tok.int(), top_logprobs=d.gather(1, tok) - log_s[:, None])
    return out


# ---------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = {}
    globals()["_prepare_" + case["op"]](case, _gen(seed), st)
    return globals()["_exact_" + case["op"]](st)


def _exact_chunk(st):
    H, kv, D, ps = st["H"], st["kv"], st["D"], st["ps"]
    G = H // kv
    out = torch.zeros(st["T"], H, D, dtype=torch.float64, device="cuda")
    starts, lens = st["starts"].tolist(), st["lens"].tolist()
    for r, total in enumerate(lens):
        first, end = starts[r], starts[r + 1]
        ids = st["tables"][r, :(total + ps - 1) // ps].long()
        for h in range(kv if end > first else 0):
            k = st["k"][0, ids, h].reshape(-1, D)[:total].double()
            v = st["v"][0, ids, h].reshape(-1, D)[:total].double()
            if "ks" in st:
                k = k * st["ks"][0, ids, h].reshape(-1, 1)[:total].double()
                v = v * st["vs"][0, ids, h].reshape(-1, 1)[:total].double()
            late = torch.triu(torch.ones(end - first, total, dtype=torch.bool, device="cuda"),
                              total - (end - first) + 1)
            for c in range(h * G, h * G + G):
                s = st["scale"] * (st["q"].view(-1, H, D)[first:end, c].double() @ k.T)
                out[first:end, c] = torch.softmax(s.masked_fill_(late, -math.inf), 1) @ v
    return out.view(st["T"], H * D)


def _exact_codes(y):
    """Values of 8-bit rows; the codes are defined by the row rounded to fp32."""
    scale = (127.0 / y.abs().amax(1).double()).float()
    q = (y * scale[:, None]).round().clamp(-127, 127)
    return {"x": q.double() / scale[:, None].double(), "scale": scale.double()}


def _exact_norm(st):
    h = st["residual"].double() + st["x"].double()
    n = h.float().double()
    length = torch.linalg.vector_norm(n, dim=1, keepdim=True)
    y = st["weight"].double() * n / torch.sqrt(length * length / st["K"] + st["eps"])
    return dict(_exact_codes(y.float()) if st["codes"] else {"y": y}, sum=h)


def _exact_gate(st):
    y = torch.sigmoid(st["gate"].double()) * st["gate"].double() * st["up"].double()
    return _exact_codes(y.float()) if st["codes"] else {"y": y}


def _exact_score(st):
    out = {"logprobs": [], "entropy": [], "top_tokens": None, "top_logprobs": []}
    for a in range(0, st["R"], 100):
        lp = torch.log_softmax(st["logits"][a:a + 100].double(), 1)
        out["logprobs"].append(lp.gather(1, st["tokens"][a:a + 100, None].long())[:, 0])
        out["entropy"].append(torch.special.entr(lp.exp()).sum(1))
        out["top_logprobs"].append(lp.sort(1, descending=True).values[:, :st["top"]]
                                   if st["top"] else None)
    return {k: torch.cat(v) if v and v[0] is not None else None for k, v in out.items()}


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once; ragged lengths at their mean."""
    op = case["op"]
    if op == "chunk":
        R, kv, D, G = case["requests"], case["kv"], case["dim"], case["group"]
        new = (case["new_lo"] + case["new_hi"]) / 2 if R > 1 else case["new_hi"]
        old = (case["old_lo"] + case["old_hi"]) / 2 if R > 1 else case["old_hi"]
        per = 2 * D * (1 if case["type"] == "int8" else 2) + (8 if case["type"] == "int8" else 0)
        return {"bytes": int(R * (new + old) * (kv * per + 4 / case["page"])
                             + R * new * kv * G * D * 8),
                "flops": int(4 * R * new * (old + (new + 1) / 2) * kv * G * D)}
    n = case["rows"] * (case["vocab"] if op == "score" else case["width"])
    if op == "score":
        return {"bytes": 4 * n + case["rows"] * (12 + 8 * case["top"]), "flops": 6 * n}
    rows = case["rows"] * 4 if case["codes"] else 0
    if op == "norm":
        return {"bytes": n * (12 + (1 if case["codes"] else 4)) + 4 * case["width"] + rows,
                "flops": 6 * n}
    return {"bytes": n * (8 + (1 if case["codes"] else 4)) + rows, "flops": 8 * n}
