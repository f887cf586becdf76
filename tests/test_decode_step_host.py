"""The cache and beam-search calls without a GPU: every refusal of the C ABI
and of the binding that is decided on the host, the size helpers, and pins of
the plain definitions that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from oracle import decode_step as ref
from ternary_weight_decoder_amd import binding as tb

NULL, SHAPE, ALIGN, WS, ALIAS = 1, 2, 3, 4, 7
A = 0x7f0000000000        # never dereferenced
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    return tb.lib()


def cache(**kw):
    c = dict(k=A, v=A + GB, k_scale=0, v_scale=0, layer_stride=1 << 20, page_stride=1 << 14,
             head_stride=1 << 13, token_stride=128, dtype=0, layers=2, pages=64, kv_heads=2,
             page_size=64, head_dim=128)
    c.update(kw)
    return tb.bitnet_kv_cache(*c.values())


BAD_CACHES = [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(dtype=2), NULL), (dict(dtype=3), SHAPE),
    (dict(dtype=-1), SHAPE), (dict(head_dim=96), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=2048), SHAPE), (dict(layers=0), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=257), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 25), SHAPE), (dict(token_stride=64), SHAPE), (dict(head_stride=1 << 31), SHAPE),
    (dict(layer_stride=1 << 40), SHAPE),
    (dict(dtype=2, k_scale=A, v_scale=A, kv_heads=256, pages=1 << 24), SHAPE),
    (dict(page_stride=(1 << 14) + 4), ALIGN), (dict(layer_stride=4), SHAPE),
    (dict(k=A + 8), ALIGN), (dict(dtype=2, k_scale=A + 2, v_scale=A), ALIGN),
    (dict(dtype=2, k_scale=A, v_scale=A, token_stride=136), ALIGN),
]


def append(L, c, layer=0, T=4, qh=12, k=A, ks=256, v=A, vs=256, slots=A, pos=A, cos=A, sin=A,
           mp=100, q=A + 2 * GB, qs=1536, qo=A + 3 * GB):
    return L.bitnet_kv_append(ctypes.byref(c), layer, T, qh, k, ks, v, vs, slots, pos, cos, sin,
                              mp, q, qs, qo, None)


def attend(L, c, layer=0, T=4, qh=12, q=A, qs=1536, tab=A, tr=4, mp=8, rows=None, lens=A,
           ml=512, out=A + GB, lse=None, ws=A + 2 * GB, wb=None):
    if wb is None:
        wb = L.bitnet_paged_attention_workspace_bytes(max(T, 1), 12, 2, 128, 512)
    return L.bitnet_paged_attention(ctypes.byref(c), layer, T, qh, q, qs, tab, tr, mp, rows, lens,
                                    ml, 0.1, out, lse, ws, wb, None)


def reorder(L, c, B=2, W=4, par=A, lens=A, ti=A, to=A + GB, mp=8):
    return L.bitnet_beam_reorder(ctypes.byref(c), B, W, par, lens, ti, to, mp, None)


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_every_cache_call_checks_the_descriptor(L, change, want):
    c = cache(**change)
    assert append(L, c) == want
    assert attend(L, c) == want
    assert reorder(L, c) == want


def test_cache_layer_out_of_range(L):
    for layer in (-1, 2):
        assert append(L, cache(), layer) == SHAPE
        assert attend(L, cache(), layer) == SHAPE
    assert L.bitnet_kv_append(None, 0, 1, 0, A, 256, A, 256, A, None, None, None, 0, None, 0, None,
                              None) == NULL


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(pos=None), NULL),
    (dict(sin=None), NULL), (dict(cos=None, sin=None), NULL), (dict(qo=None), NULL),
    (dict(q=None), NULL), (dict(T=-1), SHAPE), (dict(T=1 << 23), SHAPE), (dict(qh=0), SHAPE),
    (dict(qh=1 << 20), SHAPE), (dict(mp=0), SHAPE), (dict(ks=252), SHAPE), (dict(vs=128), SHAPE),
    (dict(qs=1532), SHAPE), (dict(ks=1 << 31), SHAPE), (dict(ks=258), ALIGN),
    (dict(qs=1538), ALIGN), (dict(k=A + 4), ALIGN), (dict(v=A + 8), ALIGN), (dict(q=A + 4), ALIGN),
    (dict(slots=A + 2), ALIGN), (dict(cos=A + 4), ALIGN), (dict(qo=A + 2 * GB + 1536), ALIAS),
    (dict(qo=A + 2 * GB, qs=1540), ALIAS), (dict(qo=A + 512), ALIAS), (dict(T=0), 0),
])
def test_append_refusals(L, kw, want):
    assert append(L, cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(tab=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(T=-1), SHAPE), (dict(T=1 << 23), SHAPE), (dict(T=5), SHAPE), (dict(qh=13), SHAPE),
    (dict(qh=0), SHAPE), (dict(qh=258, qs=1 << 16), SHAPE), (dict(qs=1280), SHAPE),
    (dict(ml=0), SHAPE), (dict(ml=513), SHAPE), (dict(mp=0), SHAPE), (dict(tr=0, rows=A), SHAPE),
    (dict(qs=1538), ALIGN), (dict(q=A + 4), ALIGN), (dict(out=A + GB + 4), ALIGN),
    (dict(rows=A + 1), ALIGN), (dict(lse=A + 2 * GB + 2), ALIGN), (dict(ws=A + 2 * GB + 16), ALIGN),
    (dict(ws=None), WS), (dict(wb=16), WS), (dict(out=A + 1024), ALIAS), (dict(lse=A + GB), ALIAS),
    (dict(ws=A + GB + 1024), ALIAS), (dict(T=0), 0),
])
def test_attention_refusals(L, kw, want):
    assert attend(L, cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(par=None), NULL), (dict(lens=None), NULL), (dict(ti=None), NULL), (dict(to=None), NULL),
    (dict(B=0), SHAPE), (dict(W=0), SHAPE), (dict(W=33), SHAPE), (dict(B=2000), SHAPE),
    (dict(B=1 << 62), SHAPE), (dict(mp=0), SHAPE), (dict(mp=1 << 25), SHAPE),
    (dict(mp=1 << 60), SHAPE), (dict(par=A + 2), ALIGN), (dict(to=A), ALIAS), (dict(to=A + 128), ALIAS),
])
def test_reorder_refusals(L, kw, want):
    assert reorder(L, cache(), **kw) == want


def pool(**kw):
    p = dict(tables=A, owned=A + GB, free_pages=A + 2 * GB, rows=4, max_pages=8, pages=32,
             page_size=16)
    p.update(kw)
    return tb.bitnet_kv_pool(*p.values())


@pytest.mark.parametrize("pk,kw,want", [
    (dict(tables=0), {}, NULL), (dict(owned=0), {}, NULL), (dict(free_pages=0), {}, NULL),
    ({}, {0: None}, NULL), ({}, {1: None}, NULL), ({}, {7: None}, NULL), (dict(rows=0), {}, SHAPE),
    (dict(rows=4097), {}, SHAPE), (dict(max_pages=0), {}, SHAPE), (dict(page_size=24), {}, SHAPE),
    (dict(max_pages=1 << 27), {}, SHAPE), (dict(pages=0), {}, SHAPE), (dict(pages=1 << 27), {}, SHAPE),
    ({}, {"T": 0}, SHAPE), ({}, {"T": 1 << 31}, SHAPE), ({}, {0: A + 3 * GB + 2}, ALIGN),
    (dict(owned=A + 64), {}, ALIAS), ({}, {2: A + 2 * GB}, ALIAS), ({}, {4: A + 8 * GB}, ALIAS),
    ({}, {2: A + 4 * GB + 4}, ALIAS),
])
def test_map_refusals(L, pk, kw, want):
    kw = dict(kw)
    T = kw.pop("T", 10)
    args = [A + (3 + i) * GB for i in range(8)]   # new, state in, state out, starts, ...
    for i, a in kw.items():
        args[i] = a
    assert L.bitnet_kv_map(ctypes.byref(pool(**pk)), T, *args, None) == want
    assert L.bitnet_kv_map(None, T, *args, None) == NULL


def select(L, B=2, W=4, V=100, x=A, ld=100, s=A + GB, f=A + 2 * GB, eos=5, so=A + 3 * GB,
           t=A + 4 * GB, p=A + 5 * GB, fo=A + 6 * GB, ws=A + 7 * GB, wb=None):
    if wb is None:
        wb = L.bitnet_beam_select_workspace_bytes(2, 4, 100)
    return L.bitnet_beam_select(B, W, V, x, ld, s, f, eos, so, t, p, fo, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(s=None), NULL), (dict(so=None), NULL), (dict(t=None), NULL),
    (dict(p=None), NULL), (dict(f=None), NULL), (dict(fo=None), NULL), (dict(B=0), SHAPE),
    (dict(W=0), SHAPE), (dict(W=33), SHAPE), (dict(B=1025), SHAPE), (dict(B=1 << 61), SHAPE),
    (dict(V=3), SHAPE), (dict(V=1 << 30, ld=1 << 30), SHAPE), (dict(ld=99), SHAPE),
    (dict(ld=1 << 31), SHAPE), (dict(eos=-1), SHAPE), (dict(eos=100), SHAPE),
    (dict(x=A + 2), ALIGN), (dict(ws=A + 7 * GB + 16), ALIGN), (dict(ws=None), WS), (dict(wb=64), WS),
    (dict(t=A + 5 * GB), ALIAS), (dict(so=A + GB + 4), ALIAS), (dict(fo=A + 2 * GB - 4), ALIAS),
    (dict(p=A + 96), ALIAS),
])
def test_select_refusals(L, kw, want):
    assert select(L, **kw) == want


def test_size_helpers(L):
    f = L.bitnet_paged_attention_workspace_bytes
    assert f(0, 12, 2, 128, 100) == 0 and f(1, 12, 5, 128, 100) == 0 and f(1, 12, 2, 100, 100) == 0
    assert f(1, 12, 2, 128, 0) == 0 and f(1, 12, 2, 128, 32768) >= 16384
    g = L.bitnet_beam_select_workspace_bytes
    assert g(1, 33, 100) == 0 and g(1, 4, 3) == 0 and g(0, 4, 100) == 0
    assert g(16, 4, 151936) >= 16384


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tb.KvCache(t, t)
    with pytest.raises(ValueError):
        tb.KvCache(t.float(), t.float())
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        tb.KvPool(8, 16, i, i, torch.zeros(8, dtype=torch.int32))


# ---- pins of the plain definitions -------------------------------------------

def test_map_definition_by_hand():
    """Three requests, pages of 4: one grows over a page, one ends, one starts."""
    tables = np.array([[7, -1, -1], [5, 6, -1], [-1, -1, -1]], np.int32)
    free = np.array([0, 1, -1, -1, -1, -1, -1, -1], np.int32)
    state = np.array([3, 8, 0, 1, 2, 0, 2], np.int32)
    o = ref.kv_map(4, 8, 12, np.array([2, -1, 5], np.int32), state, tables, tables.copy(), free)
    assert o["free"][:4].tolist() == [0, 1, 5, 6]              # 5 and 6 came back
    assert o["tables"].tolist() == [[7, 6, -1], [5, 6, -1], [5, 1, -1]]
    assert o["state"].tolist() == [5, 0, 5, 2, 0, 2, 1]
    assert o["starts"].tolist() == [0, 2, 2, 7]
    assert o["slots"].tolist() == [31, 24, 20, 21, 22, 23, 4] + [-1] * 5
    assert o["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4] + [-1] * 5
    assert o["rows"].tolist() == [0, 0, 2, 2, 2, 2, 2] + [-1] * 5
    assert o["status"].tolist() == [0, 0, 0]


def test_map_definition_refusals_by_hand():
    tables = np.full((4, 2), -1, np.int32)
    free = np.arange(8, dtype=np.int32)
    new = np.array([9, 5, 8, 1], np.int32)      # 9 > 8 tokens of a table of two pages of 4
    state = np.array([0] * 8 + [3], np.int32)
    o = ref.kv_map(4, 8, 6, new, state, tables, tables.copy(), free)
    # 5 tokens take 2 of 3 pages; 8 need 2 more; 1 needs a page: sums 4 and 5 > 3
    assert o["status"].tolist() == [1, 0, 2, 2]
    assert o["state"].tolist() == [0, 5, 0, 0, 0, 2, 0, 0, 1]
    o = ref.kv_map(4, 8, 6, new[[0, 1, 3, 2]], np.array([0] * 8 + [8], np.int32), tables,
                   tables.copy(), free)
    assert o["status"].tolist() == [1, 0, 0, 3]  # 5 + 1 tokens fill T = 6


def test_select_definition_by_hand():
    """Two beams of one group; probabilities 1/2, 1/4, 1/4 and 3/4, 1/8, 1/8."""
    x = np.log(np.array([[2, 1, 1], [6, 1, 1]], np.float64)).astype(np.float32)
    o = ref.beam_select(x, np.log(np.array([0.5, 0.25])).astype(np.float32), 2)
    np.testing.assert_allclose(np.exp(o["scores"]), [0.25, 0.1875], rtol=1e-6)
    assert o["tokens"].tolist() == [0, 0] and o["parents"].tolist() == [0, 1]
    # a finished beam keeps its score and its end token
    o = ref.beam_select(x, np.log(np.array([0.5, 0.25])).astype(np.float32), 2,
                        np.array([1, 0], np.int32), 2)
    assert o["tokens"].tolist() == [2, 0] and o["finished"].tolist() == [1, 0]
    np.testing.assert_allclose(np.exp(o["scores"]), [0.5, 0.1875], rtol=1e-6)


def test_reorder_definition_by_hand():
    """Four beams of 6 tokens, pages of 4: beam 1 has two children, 2 has two."""
    k = np.arange(8, dtype=np.float32).reshape(1, 8, 1, 1, 1) * np.ones((1, 8, 1, 4, 1), np.float32)
    tables = np.array([[0, 4], [0, 5], [0, 6], [0, 7]], np.int32)
    nk, nv, _, _, t = ref.beam_reorder(k, k, None, None, 4, np.array([1, 2, 1, 2]), [6] * 4, tables)
    assert t.tolist() == [[0, 5], [0, 6], [0, 4], [0, 7]]
    assert nk[0, :, 0, 0, 0].tolist() == [0, 1, 2, 3, 5, 5, 6, 6]   # 2 tokens copied ...
    assert nk[0, :, 0, 2, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7]   # ... and no more
    assert nv[0, 4, 0, :, 0].tolist() == [5, 5, 4, 4]


def test_outputs_inside_the_cache_are_refused(L):
    """The layer's arrays from their first to their last element; ALIAS is decided
    before the device is looked at, so where there is none a call that passes this
    check gives something else."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would run on made-up addresses")
    c = dict(k=A + 8 * GB, v=A + 16 * GB)
    last = ((63 << 14) + (1 << 13) + 63 * 128 + 127) * 2      # of a layer, bytes
    lay = 1 << 21
    for base in (8, 16):
        for layer in (0, 1):
            at = A + base * GB + layer * lay
            assert append(L, cache(**c), layer, qo=at + 1024) == ALIAS
            assert append(L, cache(**c), layer, qo=at + last - 14) == ALIAS
            assert append(L, cache(**c), layer, qo=at - 16) == ALIAS
            for kw in (dict(out=at + 4096), dict(lse=at + last - 2), dict(ws=at + 512)):
                assert attend(L, cache(**c), layer, **kw) == ALIAS, kw
            assert reorder(L, cache(**c), to=at + last - 2) == ALIAS
        # the other layer is not this call's
        assert append(L, cache(**c), 0, qo=A + base * GB + lay) != ALIAS
    assert append(L, cache(**c), 1, qo=A + 4 * GB) != ALIAS
    s = dict(c, dtype=2, k_scale=A + 24 * GB, v_scale=A + 25 * GB)
    per = 64 * 2 * 64 * 4
    for base in (24, 25):
        assert attend(L, cache(**s), 1, out=A + base * GB + 2 * per - 16) == ALIAS
        assert attend(L, cache(**s), 0, out=A + base * GB + per) != ALIAS
        assert reorder(L, cache(**s), to=A + base * GB + 2 * per - 4) == ALIAS


def test_extents_of_huge_strides_do_not_wrap(L):
    c = cache(k=A + 8 * GB, v=A + 16 * GB, page_stride=(1 << 31) - 8, pages=(1 << 24) - 1,
              page_size=128, layers=1024, layer_stride=(1 << 40) - 8)
    assert append(L, c, 0, qo=A + 64 * GB) == ALIAS
    assert reorder(L, c, to=A + 64 * GB) == ALIAS


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_scale_is_finite(L, scale):
    c = cache(k=A + 8 * GB, v=A + 16 * GB)
    ws = L.bitnet_paged_attention_workspace_bytes(4, 12, 2, 128, 512)
    assert L.bitnet_paged_attention(ctypes.byref(c), 0, 4, 12, A, 1536, A, 4, 8, None, A, 512, scale,
                                    A + GB, None, A + 2 * GB, ws, None) == SHAPE
