"""One new token whose queries are a slice of a wider row: a single row is contiguous
whatever its stride, so it may be rotated in place."""
import pytest
import torch

from tests.test_decode_step_host import A, ALIAS, GB, L, append, cache  # noqa: F401
from tests.test_gpu_decode_step import tb  # noqa: F401
from ternary_weight_decoder_amd import binding

PASSED = (5, 6)   # arguments that pass every check end at the device check without a GPU


def test_append_of_one_row_in_place(L):  # noqa: F811
    kw = dict(k=A + 4 * GB, v=A + 5 * GB, slots=A + 6 * GB, pos=A + 7 * GB, cos=A + 8 * GB, sin=A + 9 * GB)
    c = cache(k=A + 64 * GB, v=A + 80 * GB)
    for qs in (1536, 2048, 1540):
        assert append(L, c, T=1, q=A, qo=A, qs=qs, **kw) in PASSED, qs
    assert append(L, c, T=2, q=A, qo=A, qs=1536, **kw) in PASSED
    assert append(L, c, T=2, q=A, qo=A, qs=2048, **kw) == ALIAS
    assert append(L, c, T=1, q=A, qo=A + 16, qs=2048, **kw) == ALIAS


def test_stride_of_a_slice_of_one_row():
    """The stride that the calls are given for it."""
    fused = torch.zeros(1, 2048)
    assert binding._rows_stride(fused[:, :1536], 1536) == 2048
    assert binding._rows_stride(torch.zeros(2, 2048)[:1, 512:], 1536) == 2048


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.int8])
def test_append_of_one_fused_row_in_place(tb, dt):  # noqa: F811
    KV, D, H, ps, P = 2, 128, 12, 16, 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    fused = torch.randn(1, (H + 2 * KV) * D, generator=gen, device="cuda")
    cos, sin = (f(torch.arange(40.0, device="cuda")[:, None] / 100 ** (torch.arange(64.0, device="cuda") / 64))
                for f in (torch.cos, torch.sin))
    slots, positions = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (21, 37))

    def one(in_place):
        x = fused.clone()
        q, k, v = x.split([H * D, KV * D, KV * D], 1)
        pages = [torch.zeros(1, P, KV, ps, D, dtype=dt, device="cuda") for _ in range(2)]
        scales = [torch.zeros(1, P, KV, ps, device="cuda") for _ in range(2)] if dt is torch.int8 else []
        c = tb.KvCache(*pages, *scales)
        out = q if in_place else torch.empty(1, H * D, device="cuda")
        tb.bitnet_kv_append_into(c, 0, 1, H, k, v, slots, positions, cos, sin, q, out)
        return x, out.clone(), pages + scales

    apart, here = one(False), one(True)
    assert not torch.equal(apart[1], fused[:, :H * D])
    assert torch.equal(apart[1], here[1]) and torch.equal(apart[0], fused)
    assert torch.equal(here[0][:, H * D:], fused[:, H * D:])
    assert all(torch.equal(a, b) for a, b in zip(apart[2], here[2]))
    assert all(p.ne(0).any().item() for p in here[2])
