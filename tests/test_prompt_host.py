"""The calls around a prompt's projections without a GPU: every refusal of the C
ABI and of the binding that is decided on the host, the size helpers, and pins of
the plain definitions that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import decode_step, prompt as ref
from tests.test_decode_step_devices import OnDevice
from tests.test_decode_step_host import BAD_CACHES, cache
from ternary_weight_decoder_amd import binding as tb

NULL, SHAPE, ALIGN, WS, ALIAS = 1, 2, 3, 4, 7
A = 0x7f0000000000        # never dereferenced
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    return tb.lib()


# Arguments that pass every check end at the device check: there is no GPU here.
PASSED = (5, 6)


def chunk(L, c=None, layer=0, T=40, qh=12, q=A, qs=1536, R=4, st=A + GB, ln=A + 2 * GB, tab=A + 3 * GB,
          mp=8, ml=512, sc=0.1, out=A + 4 * GB, lse=None, ws=A + 5 * GB, wb=1 << 40):
    c = cache(k=A + 6 * GB, v=A + 7 * GB) if c is None else c
    return L.bitnet_chunk_attention(ctypes.byref(c), layer, T, qh, q, qs, R, st, ln, tab, mp, ml, sc,
                                    out, lse, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(st=None), NULL), (dict(ln=None), NULL), (dict(tab=None), NULL),
    (dict(out=None), NULL), (dict(T=-1), SHAPE), (dict(T=1 << 23), SHAPE), (dict(qh=0), SHAPE),
    (dict(qh=13), SHAPE), (dict(qh=130), SHAPE), (dict(R=0), SHAPE), (dict(R=4097), SHAPE),
    (dict(mp=0), SHAPE), (dict(ml=0), SHAPE), (dict(ml=513), SHAPE), (dict(ml=1 << 30, mp=1 << 25), SHAPE),
    (dict(qs=1532), SHAPE), (dict(qs=1 << 31), SHAPE), (dict(sc=math.inf), SHAPE),
    (dict(sc=math.nan), SHAPE), (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE),
    (dict(T=(1 << 23) - 1, qh=128, qs=16384, ml=(1 << 30) - 1, mp=1 << 25), SHAPE),   # 2^52 places
    (dict(qs=1538), ALIGN), (dict(q=A + 4), ALIGN), (dict(out=A + 4 * GB + 8), ALIGN),
    (dict(st=A + GB + 2), ALIGN), (dict(ln=A + 2 * GB + 1), ALIGN), (dict(tab=A + 3 * GB + 2), ALIGN),
    (dict(lse=A + 8 * GB + 2), ALIGN), (dict(ws=A + 5 * GB + 128), ALIGN), (dict(ws=None), WS),
    (dict(wb=100), WS),
    (dict(out=A), ALIAS), (dict(out=A + 39 * 6144), ALIAS), (dict(lse=A + 4 * GB), ALIAS),
    (dict(lse=A), ALIAS), (dict(ws=A), ALIAS), (dict(out=A + GB), ALIAS), (dict(lse=A + 2 * GB), ALIAS),
    (dict(out=A + 3 * GB), ALIAS), (dict(out=A + 6 * GB), ALIAS), (dict(ws=A + 7 * GB), ALIAS),
    (dict(lse=A + 6 * GB + 1024), ALIAS),
])
def test_chunk_refusals(L, kw, want):
    assert chunk(L, **kw) == want


def test_chunk_passes_and_empty(L):
    assert chunk(L) in PASSED
    assert chunk(L, T=0) == 0
    assert chunk(L, lse=A + 8 * GB, R=4096) in PASSED


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_chunk_bad_caches(L, kw, want):
    assert chunk(L, cache(**kw)) == want


def test_chunk_workspace(L):
    f = L.bitnet_chunk_attention_workspace_bytes
    assert f(40, 4, 12, 2, 128, 512) > 0
    for bad in ((0, 4, 12, 2, 128, 512), (40, 0, 12, 2, 128, 512), (40, 4, 13, 2, 128, 512),
                (40, 4, 12, 2, 96, 512), (40, 4, 12, 2, 128, 0), (40, 4097, 12, 2, 128, 512),
                ((1 << 23) - 1, 1, 128, 2, 128, (1 << 30) - 1)):
        assert f(*bad) == 0
    # bounded, whatever the lengths
    assert f(1 << 20, 4096, 64, 8, 256, 1 << 20) < 1 << 28
    need = f(40, 4, 12, 2, 128, 512)
    assert chunk(L, wb=need) in PASSED and chunk(L, wb=need - 1) == WS


def norm(L, M=4, K=64, x=A, xs=64, r=A + GB, rs=64, w=A + 2 * GB, eps=1e-6, s=A + 3 * GB,
         y=A + 4 * GB, xq=A + 5 * GB, sc=A + 6 * GB):
    return L.bitnet_add_rms_norm(M, K, x, xs, r, rs, w, eps, s, y, xq, sc, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None, xq=None, sc=None), NULL),
    (dict(xq=None), NULL), (dict(sc=None), NULL), (dict(M=-1), SHAPE), (dict(M=1 << 23), SHAPE),
    (dict(K=0), SHAPE), (dict(K=62), SHAPE), (dict(K=32772, xs=40000, rs=40000), SHAPE),
    (dict(xs=60), SHAPE), (dict(rs=60), SHAPE), (dict(xs=1 << 31), SHAPE), (dict(rs=1 << 31), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=math.inf), SHAPE), (dict(eps=math.nan), SHAPE),
    (dict(xs=66), ALIGN), (dict(rs=66), ALIGN), (dict(x=A + 4), ALIGN), (dict(r=A + GB + 8), ALIGN),
    (dict(w=A + 2 * GB + 4), ALIGN), (dict(s=A + 3 * GB + 4), ALIGN), (dict(y=A + 4 * GB + 4), ALIGN),
    (dict(xq=A + 5 * GB + 4), ALIGN), (dict(sc=A + 6 * GB + 2), ALIGN),
    (dict(y=A), ALIAS), (dict(y=A + GB + 3 * 256), ALIAS), (dict(y=A + 2 * GB), ALIAS),
    (dict(s=A + 4 * GB), ALIAS), (dict(xq=A + 4 * GB + 256), ALIAS), (dict(sc=A + 5 * GB), ALIAS),
    (dict(xq=A), ALIAS), (dict(sc=A + 2 * GB), ALIAS), (dict(s=A + 16), ALIAS),
    (dict(s=A, xs=68), ALIAS), (dict(s=A + GB, rs=68), ALIAS), (dict(s=A + 2 * GB), ALIAS),
])
def test_norm_refusals(L, kw, want):
    assert norm(L, **kw) == want


def test_norm_passes(L):
    for kw in (dict(), dict(s=A), dict(s=A + GB), dict(r=None, rs=0), dict(s=None), dict(y=None),
               dict(xq=None, sc=None), dict(r=A), dict(xs=68, rs=72), dict(eps=0.0),
               dict(K=32768, xs=32768, rs=32768), dict(M=(1 << 23) - 1, r=A, s=A, y=A + 8 * GB,
                                                       xq=None, sc=None)):
        assert norm(L, **kw) in PASSED, kw
    assert norm(L, M=0) == 0


def test_one_row_in_place_whatever_its_stride(L):
    """A single row is contiguous."""
    for kw in (dict(s=A, xs=68), dict(s=A + GB, rs=128)):
        assert norm(L, M=1, **kw) in PASSED and norm(L, M=2, **kw) == ALIAS
    for kw in (dict(y=A, gs=68), dict(y=A + GB, us=128)):
        assert gate(L, M=1, **kw) in PASSED and gate(L, M=2, **kw) == ALIAS


def gate(L, M=4, K=64, g=A, gs=64, u=A + GB, us=64, y=A + 2 * GB, xq=A + 3 * GB, sc=A + 4 * GB):
    return L.bitnet_silu_mul(M, K, g, gs, u, us, y, xq, sc, None)


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), NULL), (dict(u=None), NULL), (dict(y=None, xq=None, sc=None), NULL),
    (dict(xq=None), NULL), (dict(sc=None), NULL), (dict(M=-1), SHAPE), (dict(K=66), SHAPE),
    (dict(K=0), SHAPE), (dict(gs=60), SHAPE), (dict(us=1 << 31), SHAPE), (dict(gs=70), ALIGN),
    (dict(us=65), ALIGN), (dict(g=A + 8), ALIGN), (dict(u=A + GB + 4), ALIGN),
    (dict(y=A + 2 * GB + 8), ALIGN), (dict(xq=A + 3 * GB + 8), ALIGN), (dict(sc=A + 4 * GB + 1), ALIGN),
    (dict(y=A + 16), ALIAS), (dict(y=A, gs=68), ALIAS), (dict(y=A + GB, us=68), ALIAS),
    (dict(xq=A), ALIAS), (dict(sc=A + GB), ALIAS), (dict(xq=A + 2 * GB), ALIAS),
    (dict(sc=A + 3 * GB), ALIAS),
])
def test_gate_refusals(L, kw, want):
    assert gate(L, **kw) == want


def test_gate_passes(L):
    for kw in (dict(), dict(y=A), dict(y=A + GB), dict(u=A), dict(xq=None, sc=None), dict(y=None),
               dict(u=A + 256, gs=128, us=128)):
        assert gate(L, **kw) in PASSED, kw
    assert gate(L, M=0) == 0


def score(L, R=4, V=100, x=A, ld=100, tok=A + GB, top=5, lp=A + 2 * GB, e=A + 3 * GB, tt=A + 4 * GB,
          tl=A + 5 * GB, ws=A + 6 * GB, wb=1 << 40):
    return L.bitnet_token_logprobs(R, V, x, ld, tok, top, lp, e, tt, tl, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(tok=None), NULL), (dict(lp=None), NULL), (dict(tt=None), NULL),
    (dict(tl=None), NULL), (dict(top=0), NULL), (dict(top=0, tt=None), NULL),
    (dict(tok=None, lp=None, e=None, top=0, tt=None, tl=None), NULL),
    (dict(R=-1), SHAPE), (dict(R=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=4), SHAPE),
    (dict(V=1 << 30, ld=1 << 30), SHAPE), (dict(ld=99), SHAPE), (dict(ld=1 << 31), SHAPE),
    (dict(top=33), SHAPE), (dict(top=-1, tt=None, tl=None), SHAPE),
    (dict(x=A + 2), ALIGN), (dict(tok=A + GB + 1), ALIGN), (dict(lp=A + 2 * GB + 2), ALIGN),
    (dict(e=A + 3 * GB + 2), ALIGN), (dict(tt=A + 4 * GB + 2), ALIGN), (dict(tl=A + 5 * GB + 2), ALIGN),
    (dict(ws=A + 6 * GB + 64), ALIGN), (dict(ws=None), WS), (dict(wb=1000), WS),
    (dict(lp=A), ALIAS), (dict(e=A + 2 * GB + 12), ALIAS), (dict(tt=A + 5 * GB), ALIAS),
    (dict(tl=A + GB), ALIAS), (dict(ws=A), ALIAS), (dict(lp=A + 6 * GB), ALIAS), (dict(e=A + GB), ALIAS),
])
def test_score_refusals(L, kw, want):
    assert score(L, **kw) == want


def test_score_passes_and_workspace(L):
    for kw in (dict(), dict(top=0, tt=None, tl=None), dict(tok=None, lp=None), dict(e=None),
               dict(e=None, tok=None, lp=None), dict(R=65535), dict(ld=103, x=A + 4)):
        assert score(L, **kw) in PASSED, kw
    assert score(L, R=0) == 0
    f = L.bitnet_token_logprobs_workspace_bytes
    assert f(4, 100, 5) > 0 and f(0, 100, 5) == 0 and f(4, 100, 101) == 0 and f(4, 100, 33) == 0
    assert f(65535, 1 << 20, 32) < 1 << 28
    need = f(4, 100, 5)
    assert score(L, wb=need) in PASSED and score(L, wb=need - 1) == WS


# ---- the binding's own checks (stand-ins for device tensors) --------------------

def stand_ins(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = tb.KvCache(*(OnDevice(0, 1, 4, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    f = lambda *s: OnDevice(0, *s, dtype=torch.float32)
    return c, f, lambda *s: OnDevice(0, *s)


def test_binding_refusals(monkeypatch):
    c, f, i = stand_ins(monkeypatch)
    bad = [
        lambda: tb.bitnet_chunk_attention(c, 0, f(6, 100), i(4), i(3), i(3, 2)),
        lambda: tb.bitnet_chunk_attention(c, 0, f(6, 256), i(3), i(3), i(3, 2)),
        lambda: tb.bitnet_chunk_attention(c, 0, f(6, 256), i(4), i(4), i(3, 2)),
        lambda: tb.bitnet_chunk_attention(c, 0, f(6, 256), i(4), i(3), i(6)),
        lambda: tb.bitnet_chunk_attention(c, 0, f(6, 256), f(4), i(3), i(3, 2)),
        lambda: tb.bitnet_chunk_attention(c, 0, i(6, 256), i(4), i(3), i(3, 2)),
        lambda: tb.bitnet_chunk_attention(c, 0, OnDevice(1, 6, 256, dtype=torch.float32), i(4), i(3),
                                          i(3, 2)),
        lambda: tb.bitnet_add_rms_norm(f(4, 64), f(65)),
        lambda: tb.bitnet_add_rms_norm(f(4, 64), f(64), residual=f(4, 68)),
        lambda: tb.bitnet_add_rms_norm(i(4, 64), f(64)),
        lambda: tb.bitnet_add_rms_norm(f(4, 64), OnDevice(1, 64, dtype=torch.float32)),
        lambda: tb.bitnet_silu_mul(f(4, 64), f(4, 68)),
        lambda: tb.bitnet_silu_mul(f(4, 64), i(4, 64)),
        lambda: tb.bitnet_token_logprobs(f(4, 100), i(5)),
        lambda: tb.bitnet_token_logprobs(f(4, 100), f(4)),
        lambda: tb.bitnet_token_logprobs(i(4, 100)),
        lambda: tb.bitnet_token_logprobs(torch.zeros(4, 100)),
        lambda: tb.bitnet_silu_mul(torch.zeros(4, 64), torch.zeros(4, 64)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", n)


def test_stream_of_another_device(monkeypatch):
    from types import SimpleNamespace
    c, f, i = stand_ins(monkeypatch)
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for call in (lambda s: tb.bitnet_chunk_attention(c, 0, f(6, 256), i(4), i(3), i(3, 2), stream=s),
                 lambda s: tb.bitnet_add_rms_norm(f(4, 64), f(64), stream=s),
                 lambda s: tb.bitnet_silu_mul(f(4, 64), f(4, 64), stream=s),
                 lambda s: tb.bitnet_token_logprobs(f(4, 100), stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(other)


def test_rows_strides():
    """The stride that the calls are given: a tensor's own, but for a single row,
    whose stride means nothing."""
    x = torch.zeros(6, 40)
    assert tb._rows_stride(x, 40) == 40 and tb._rows_stride(x[:, :30], 30) == 40
    assert tb._rows_stride(x[:1], 40) == 40 and tb._rows_stride(x[:1, :30], 30) in (30, 40)
    assert tb._rows_stride(torch.zeros(3, 41)[:, :40], 40) == 41
    assert tb._rows_stride(torch.zeros(1, 41)[:, :40], 40) == 40
    assert tb._rows_stride(torch.zeros(1).expand(1, 1), 1) == 4
    assert tb._rows_stride(torch.empty_strided((1, 8), (1 << 31, 1), device="meta"), 8) == 8
    assert tb._rows_stride(torch.empty_strided((1, 8), (3, 1), device="meta"), 8) == 8
    assert tb._rows_stride(torch.empty_strided((2, 8), (0, 1), device="meta"), 8) == 0   # refused later


# ---- pins of the plain definitions ----------------------------------------------

def test_pin_request_rows():
    assert ref.request_rows(5, [0, 2, 2, 5], [7, 9, 3], 100) == [
        (0, 0, 6), (0, 1, 7), (2, 2, 1), (2, 3, 2), (2, 4, 3)]
    # lengths shorter than what is new, out of range, starts that fall or pass T
    assert ref.request_rows(4, [1, 3, 2, 9], [1, 5, 200], 6) == [(0, 1, 0), (0, 2, 1), (2, 3, 6)]
    assert ref.request_rows(2, [-4, 1, 2], [-5, 0], 6) == [(0, 0, 0), (1, 1, 0)]


def test_pin_chunk_attention():
    """Two tokens: the first sees itself, the second weighs both by softmax."""
    q = np.array([[[1.0]], [[2.0]]], np.float32)
    k, v = np.array([[[0.0], [math.log(3) / 2]]]), np.array([[[1.0], [5.0]]])
    got = ref.chunk_attention(q, [0, 2], [2], 2, lambda r, n: k[:, :n], lambda r, n: v[:, :n], 1.0)
    assert got[0][0] == 1.0 and got[0][1] == 0.0
    assert math.isclose(got[1][0].item(), 0.25 * 1 + 0.75 * 5) and math.isclose(got[1][1].item(), math.log(4))
    out, lse, *_ = decode_step.attention(q[1], k, v, 1.0)
    assert out == got[1][0] and lse == got[1][1]


def test_pin_rows():
    h, y = ref.add_rms_norm(np.array([[3.0, 4.0], [0.0, 0.0]], np.float32), np.float32([1, 2]), 0.0,
                            np.array([[0.0, 0.0], [0.0, 0.0]], np.float32))
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)], [0, 0]]) and (h == [[3, 4], [0, 0]]).all()
    q, s = ref.quant_rows(np.float32([[1.0, -0.5, 0.25], [0, 0, 0]]))
    assert q.tolist() == [[127, -64, 32], [0, 0, 0]] and s.tolist() == [127.0, 1.0]   # -63.5, 31.75
    assert np.allclose(ref.silu_mul(np.float32([0, math.log(3), -800]), np.float32([5, 2, 1])),
                       [0, 2 * math.log(3) * 0.75, 0])


def test_pin_logprobs():
    x = np.log(np.float64([[1, 2, 1, 4]])).astype(np.float32)
    x[0, 2] = x[0, 0]
    w = ref.token_logprobs(x, [1], 3)
    assert np.allclose(w["logprobs"], math.log(2 / 8)) and w["top_tokens"].tolist() == [[3, 1, 0]]
    p = np.float64([1, 2, 1, 4]) / 8
    assert np.allclose(w["entropy"], -(p * np.log(p)).sum())
    none = ref.token_logprobs(np.full((1, 3), -np.inf, np.float32), [2], 2)
    assert none["logprobs"][0] == -np.inf and none["entropy"][0] == 0 and none["top_tokens"].tolist() == [[0, 1]]
    assert ref.token_logprobs(x, [-1])["logprobs"][0] == 0
