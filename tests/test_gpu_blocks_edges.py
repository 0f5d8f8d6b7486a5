"""GPU parity of the write into the INT8 cache at the ends of its scales, bit for bit against the oracle."""

import numpy as np
import pytest

import dequant_gemv_w4_amd as w4
from test_gpu_blocks import Cache, dev

pytestmark = pytest.mark.gpu
LEAST = np.float32(2.0 ** -93 / 127)                          # of the scales that a write leaves


@pytest.mark.parametrize("old", [np.float32(2.0 ** -100), np.float32(1.005 * 2.0 ** -100), np.nextafter(LEAST, np.float32(0)), LEAST,
                                 np.nextafter(LEAST, np.float32(1))])
@pytest.mark.parametrize("rows", [[5], [3, 4, 15], [0, 1]])
@pytest.mark.parametrize("d", [64, 128])
def test_values_below_the_least_step_keep_their_sign(d, rows, old):
    # a cache made elsewhere under a scale that no write leaves, and values just below the least that counts: 128 steps of it
    kv = 2
    c = Cache(1, kv, 16, d, seed=d)
    for n, s in (("k", c.gpu.k_scales), ("v", c.gpu.v_scales)):
        c.scales[n][:] = old
        s.fill_(float(old))
    rng = np.random.default_rng(len(rows))
    x = (rng.choice([1.0, -1.0, 0.5], (len(rows), 2 * kv * d)) * (2.0 ** -93 * (1 - 2.0 ** -20))).astype(np.float32)
    w4.w4_cache_write(dev(x), c.gpu, dev(np.array(rows, np.int64)))
    x3 = x.reshape(len(rows), -1, d)
    for i, (codes, scales) in enumerate(((c.gpu.k, c.gpu.k_scales), (c.gpu.v, c.gpu.v_scales))):
        got = codes.cpu().numpy()[0][:, rows].transpose(1, 0, 2).astype(np.float64)
        y = x3[:, i * kv: (i + 1) * kv].astype(np.float64)
        step = float(scales.cpu().numpy().max())
        assert np.all(got * np.sign(y) >= 0)
        # within half a step, or zeros where nothing is left of the block
        assert np.all(np.abs(got * step - y) <= step * (0.5 + 127 * 2.0 ** -23)) or (step == 0 and not got.any())
    assert c.write(x3, 0, rows) == 0
    c.same(f"old {old} rows {rows}")
