"""The 4-bit store at the ends of its parameters' range: bf16 groups whose minimum lies past the
largest fp16 number, so that it is clamped and codes have to be clamped too. Bit for bit."""
import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

# minimum and range of a group: minima inside, at and past +-65504, scales from below 128 to past 65504
LOWS = [-3e38, -9e5, -1e5, -8e4, -7e4, -65792.0, -65536.0, -65280.0, 65280.0, 65536.0, 7e4, 1e5, 9e5, 3e38]
RANGES = [0.0, 1e3, 1.8e3, 2e3, 1e4, 7e4, 2e5, 9e5, 9.9e5, 2e6, 3e38]


@pytest.mark.parametrize("D", [64, 128])
def test_append_minima_past_fp16(D):
    rng = np.random.default_rng(D)
    NG = D // 32
    groups = []
    for low in LOWS:
        for r in RANGES:
            x = low + r * rng.random(32)
            x[rng.integers(32)] = low
            groups.append(x)
    x = np.zeros(32)
    x[7] = -1e5                                      # one far element among small ones
    groups.append(x + rng.normal(0, 1, 32))
    # ordinary groups beside them: rows of one far group and NG - 1 near ones
    T = len(groups)
    k = rng.normal(0, 1, (T, 2, NG, 32))
    for i, x in enumerate(groups):
        k[i, 0, i % NG] = x
        k[i, 1, -1 - i % NG] = -x[::-1]
    k = torch.from_numpy(k.reshape(T, 2, D)).float().clamp(-3.3e38, 3.3e38).bfloat16()
    v = k.flip(0).contiguous()
    c = b.Q4Cache.empty(-(-T // 16), 2, 16, D, torch.bfloat16)
    arrays = [t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_params, c.v_params)]
    want = O.q4_append(k.float().numpy(), v.float().numpy(), np.arange(T), *arrays)
    b.append_q4(k.cuda(), v.cuda(), torch.arange(T, device="cuda"), c)
    assert b.get_error() == 0
    for g, w in zip((c.k_codes, c.v_codes, c.k_params, c.v_params), want):
        np.testing.assert_array_equal(g.cpu().numpy().view(np.uint8), w.view(np.uint8))
