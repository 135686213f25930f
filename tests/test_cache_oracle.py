"""The cache oracle's own pins, and its numbers against torch's conversions."""
import numpy as np
import torch

import cache_oracle as co


def test_codes_against_torch():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c.copy()).view(torch.float8_e4m3fn).double().numpy()
    got = co.value(c, "e4m3")
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    rng = np.random.default_rng(0)
    mids = np.concatenate([co._MIDDLES, -co._MIDDLES, co._E4M3[:127], [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11]])
    x = np.concatenate([mids, rng.uniform(-448, 448, 4000), rng.normal(0, 0.02, 4000)]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(co.code(x.astype(np.float64), "e4m3"), want)
    assert np.array_equal(co.code([1e9, -np.inf, 448.0, np.nan], "e4m3"), [0x7e, 0xfe, 0x7e, 0x7f])
    assert np.array_equal(co.code([0.5, 1.5, -2.5, 127.4, -1e9, np.nan], "int8").view(np.int8), [0, 2, -2, 127, -127, 0])


def test_layout_round_trip():
    rng = np.random.default_rng(1)
    k, v = (rng.integers(0, 256, (2, 3, 32, 64), dtype=np.uint8) for _ in range(2))
    ks, vs = co.to_stored(k, v)
    assert ks.shape == (2, 3, 2, 4, 16, 16) and vs.shape == (2, 3, 2, 64, 16)
    assert ks[1, 2, 1, 3, 5, 7] == k[1, 2, 21, 55] and vs[1, 2, 1, 55, 5] == v[1, 2, 21, 55]
    k2, v2 = co.from_stored(ks, vs)
    assert np.array_equal(k, k2) and np.array_equal(v, v2)
