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
