"""Inputs of the calls that write the cache, held against what they write, and the
parts of a strided cache that are not its own.  Addresses are made up: ALIAS is
decided before the device is looked at, so where there is none a call that passes
this check gives something else."""
import ctypes

import numpy as np
import pytest

from tests.test_decode_step_host import A, ALIAS, GB, L, append, cache, reorder  # noqa: F401

FAR = A + 64 * GB


@pytest.fixture(autouse=True)
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would run on made-up addresses")


def inputs(**kw):
    """Arguments of an append whose arrays are far from the cache and apart."""
    names = ("k", "v", "slots", "pos", "cos", "sin", "q", "qo")
    a = {n: FAR + i * GB for i, n in enumerate(names)}
    a.update(kw)
    return a


def plain(**kw):
    return cache(k=A + 8 * GB, v=A + 16 * GB, **kw)


LAST = ((63 << 14) + (1 << 13) + 63 * 128 + 127) * 2      # of a layer, bytes


@pytest.mark.parametrize("name,size", [("k", (3 * 256 + 256) * 4), ("v", 4 * 256 * 4), ("slots", 16),
                                       ("pos", 16), ("cos", 100 * 64 * 4), ("sin", 100 * 64 * 4),
                                       ("q", 4 * 1536 * 4)])
def test_append_inputs_inside_the_layer(L, name, size):  # noqa: F811
    c, lay = plain(), 1 << 21
    assert append(L, c, **inputs()) != ALIAS
    for base in (8, 16):
        for layer in (0, 1):
            at = A + base * GB + layer * lay
            for where in (at, at + 4096, at + LAST - 14, at - size + 16):
                assert append(L, c, layer, **inputs(**{name: where})) == ALIAS, (base, layer, where - at)
            assert append(L, c, layer, **inputs(**{name: at - size - lay * layer})) != ALIAS
            assert append(L, c, layer, **inputs(**{name: at + 2 * lay})) != ALIAS
        # the other layer is read and written by nobody here
        assert append(L, c, 0, **inputs(**{name: A + base * GB + lay})) != ALIAS


def test_append_of_eight_bits_inputs_inside_the_scales(L):  # noqa: F811
    c = cache(k=A + 8 * GB, v=A + 16 * GB, dtype=2, k_scale=A + 24 * GB, v_scale=A + 25 * GB)
    per = 64 * 2 * 64 * 4
    for base in (24, 25):
        for name in ("k", "slots", "q"):
            assert append(L, c, 1, **inputs(**{name: A + base * GB + per})) == ALIAS
            assert append(L, c, 1, **inputs(**{name: A + base * GB + 2 * per - 16})) == ALIAS
            assert append(L, c, 1, **inputs(**{name: A + base * GB + 2 * per})) != ALIAS
    # arrays that the call does not use are not looked at
    assert append(L, c, 0, **inputs(pos=A + 8 * GB, cos=None, sin=None, q=None, qo=None)) != ALIAS


@pytest.mark.parametrize("name", ["par", "lens", "ti"])
def test_reorder_inputs_inside_the_cache(L, name):  # noqa: F811
    a = dict(par=FAR, lens=FAR + GB, ti=FAR + 2 * GB, to=FAR + 3 * GB)
    c = plain()
    assert reorder(L, c, **a) != ALIAS
    for base in (8, 16):
        for layer in (0, 1):
            at = A + base * GB + layer * (1 << 21)
            for where in (at, at + 4096, at + LAST - 2):
                assert reorder(L, c, **{**a, name: where}) == ALIAS
    s = cache(k=A + 8 * GB, v=A + 16 * GB, dtype=2, k_scale=A + 24 * GB, v_scale=A + 25 * GB)
    assert reorder(L, s, **{**a, name: A + 25 * GB + 1024}) == ALIAS


def test_what_lies_between_the_rows_of_a_strided_cache_passes(L):  # noqa: F811
    """Rows of 128 channels 192 apart, a page's heads 16384 apart: inputs in the 64
    elements behind a row and in the room behind a head's tokens are not the
    cache's, and one element further they are."""
    c = plain(token_stride=192, head_stride=1 << 14, page_stride=1 << 15, layer_stride=1 << 21)
    for base in (8, 16):
        for layer, page, head, tok in ((0, 0, 0, 0), (1, 3, 1, 62), (0, 63, 1, 5), (1, 63, 0, 0)):
            row = A + base * GB + 2 * ((layer << 21) + (page << 15) + (head << 14) + tok * 192)
            assert append(L, c, layer, T=1, **inputs(slots=row + 256)) != ALIAS
            assert append(L, c, layer, T=1, **inputs(slots=row + 380)) != ALIAS
            assert append(L, c, layer, T=1, **inputs(slots=row + 252)) == ALIAS
            assert append(L, c, layer, T=32, **inputs(slots=row + 256)) != ALIAS      # 128 bytes
            assert append(L, c, layer, T=33, **inputs(slots=row + 256)) == ALIAS
            behind = A + base * GB + 2 * ((layer << 21) + (page << 15) + (head << 14) + 63 * 192 + 128)
            room = 2 * ((1 << 14) - 63 * 192 - 128)
            last = page == 63 and head == 1
            assert append(L, c, layer, T=room // 4, **inputs(slots=behind)) != ALIAS
            assert append(L, c, layer, T=room // 4 + 1, **inputs(slots=behind)) == (
                ALIAS if not last else append(L, c, layer, T=room // 4, **inputs(slots=behind)))


def test_against_a_map_of_the_bytes(L):  # noqa: F811
    """Small caches in random strides and orders against a map of their bytes."""
    rng = np.random.default_rng(0)
    D, es = 64, 2
    for trial in range(40):
        n = {"layer": int(rng.integers(1, 4)), "page": int(rng.integers(1, 5)),
             "head": int(rng.integers(1, 4)), "token": int(2 ** rng.integers(0, 4))}
        order = list(n)
        rng.shuffle(order)
        stride, span = {}, D
        for d in order:                                   # the innermost first
            stride[d] = span + 8 * int(rng.integers(0, 20))
            span = (n[d] - 1) * stride[d] + span
        c = cache(k=FAR - 4 * GB, v=FAR - 2 * GB, layers=n["layer"], pages=n["page"],
                  kv_heads=n["head"], page_size=n["token"], head_dim=D, layer_stride=stride["layer"],
                  page_stride=stride["page"], head_stride=stride["head"],
                  token_stride=stride["token"])
        i = np.indices([n[d] for d in ("layer", "page", "head", "token")]).reshape(4, -1)
        at = sum(i[j] * stride[d] for j, d in enumerate(("layer", "page", "head", "token")))
        whole = np.zeros(span * es + 4096, bool)
        own = [whole.copy() for _ in range(n["layer"])]
        for layer, a in zip(i[0], at):
            own[layer][a * es:(a + D) * es] = True
            whole[a * es:(a + D) * es] = True
        for _ in range(60):
            x, T = 4 * int(rng.integers(0, span * es // 4 + 64)), int(rng.integers(1, 40))
            layer = int(rng.integers(0, n["layer"]))
            base = int(rng.choice([FAR - 4 * GB, FAR - 2 * GB]))
            rows = inputs(k=FAR + 20 * GB, v=FAR + 21 * GB, ks=256, vs=256, slots=base + x, pos=None,
                          cos=None, sin=None, q=None, qo=None)
            got = append(L, c, layer, T=T, **rows)
            assert (got == ALIAS) == own[layer][x:x + 4 * T].any(), (trial, n, stride, order, x, T)
            got = L.bitnet_beam_reorder(ctypes.byref(c), 1, min(T, 32), FAR, base + x, FAR + GB,
                                        FAR + 2 * GB, 4, None)
            assert (got == ALIAS) == whole[x:x + 4 * min(T, 32)].any(), (trial, n, stride, order, x, T)
