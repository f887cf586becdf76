"""Norm and gated activation whose fp32 rows overflow, though the inputs are finite:
scale and codes are those of the quantization of the call's fp32 row all the same."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import dev, say, tb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [128, 640, 1536, 8960, 12032])
def test_rows_that_overflow(tb, K):  # noqa: F811
    import torch
    say(f"[rows] overflow {K}")
    rng = np.random.default_rng(K)
    x = rng.normal(0, 1, (9, K)).astype(np.float32)
    x[:, ::7] = 0
    big = np.ones(K, np.float32)
    big[rng.choice(K, 5, replace=False)] = 3e38
    huge = x * np.float32(1e20)
    huge[4:6] = x[4:6]              # rows that do not, among them
    up = huge * np.sign(rng.normal(0, 1, K)).astype(np.float32)
    for call in (lambda c: tb.bitnet_add_rms_norm(dev(x), dev(big), 1e-6, codes=c),
                 lambda c: tb.bitnet_silu_mul(dev(np.abs(huge)), dev(up), codes=c)):
        a, b = call(False)["y"], call(True)
        q, s = tb.bitnet_quant_act(a)
        assert torch.isinf(a).any() and (s == 0).any()
        assert torch.equal(s, b["x_scale"]) and torch.equal(q, b["xq"])
