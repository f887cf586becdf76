"""Arrays of one pool or cache on different devices are refused (stand-ins for
tensors: there need not be two devices, or one)."""
import pytest
import torch

from ternary_weight_decoder_amd import binding as tb


class OnDevice:
    """What the checks look at."""

    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.int32):
        self.device, self.shape, self.dtype = torch.device("cuda", device), torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        st = torch.empty(self.shape, device="meta").stride()
        return st if i is None else st[i]

    def data_ptr(self):
        return 0x7f0000000000


@pytest.mark.parametrize("devices", [(0, 1, 0), (0, 0, 1), (1, 0, 0)])
def test_pool_of_two_devices(devices):
    t, o, f = devices
    with pytest.raises(ValueError, match="device"):
        tb.KvPool(8, 16, OnDevice(t, 2, 4), OnDevice(o, 2, 4), OnDevice(f, 8))


def test_pool_of_one_device():
    for d in (0, 1):
        pool = tb.KvPool(8, 16, OnDevice(d, 2, 4), OnDevice(d, 2, 4), OnDevice(d, 8))
        assert (pool.rows, pool.max_pages) == (2, 4)


@pytest.mark.parametrize("devices", [(0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)])
def test_cache_of_two_devices(devices):
    shape = (1, 4, 2, 16, 64)
    k, v = (OnDevice(d, *shape, dtype=torch.int8) for d in devices[:2])
    ks, vs = (OnDevice(d, *shape[:4], dtype=torch.float32) for d in devices[2:])
    with pytest.raises(ValueError):
        tb.KvCache(k, v, ks, vs)
    ok = [OnDevice(1, *shape, dtype=torch.int8) for _ in range(2)] + [
        OnDevice(1, *shape[:4], dtype=torch.float32) for _ in range(2)]
    assert tb.KvCache(*ok).kv_heads == 2


def test_stream_of_another_device(monkeypatch):
    """Each call refuses a stream that is not of its tensors' device, before it
    allocates or launches anything."""
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    shape = (1, 4, 2, 16, 64)
    cache = tb.KvCache(*(OnDevice(0, *shape, dtype=torch.bfloat16) for _ in range(2)))
    pool = tb.KvPool(8, 16, OnDevice(0, 2, 4), OnDevice(0, 2, 4), OnDevice(0, 8))
    f32 = lambda *s: OnDevice(0, *s, dtype=torch.float32)
    i32 = lambda *s: OnDevice(0, *s)
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for call in (lambda s: tb.bitnet_kv_map(pool, 4, i32(2), i32(5), stream=s),
                 lambda s: tb.bitnet_kv_append(cache, 0, f32(3, 128), f32(3, 128), i32(3), stream=s),
                 lambda s: tb.bitnet_paged_attention(cache, 0, f32(2, 128), i32(2, 4), i32(2), stream=s),
                 lambda s: tb.bitnet_beam_select(f32(4, 100), f32(4), 2, stream=s),
                 lambda s: tb.bitnet_beam_reorder(cache, i32(4, 4), i32(4), i32(4), 2, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(other)
