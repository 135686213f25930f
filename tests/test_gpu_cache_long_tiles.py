"""Prompts behind long contexts, through the kernel that shares positions
between four waves: dozens of steps, so that both of its buffers are filled and
read many times.  Rows picked from all over the call, against 64 bits."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, HALF, SMALLEST, Setup, ltc  # noqa: F401

pytestmark = pytest.mark.gpu

# heads, group, dim, page, codes, dtype, rows and positions before them of each sequence
SHAPES = {
    "64": (4, 16, 64, 16, "e4m3", BF, [513, 499], [2101, 1800]),
    "96 int8": (5, 13, 96, 32, "int8", FP, [700, 0, 333], [1700, 100, 2777]),
    "128": (4, 16, 128, 64, "e4m3", FP, [1030], [2900]),
    "128 int8": (16, 4, 128, 256, "int8", BF, [997], [3001]),
    "192": (8, 4, 192, 64, "e4m3", BF, [1001], [2500]),
    "256": (4, 8, 256, 128, "e4m3", FP, [1100], [1999]),
    "256 int8": (3, 11, 256, 16, "int8", BF, [640, 501], [2600, 1300]),
}


@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("name", list(SHAPES))
def test_attend(ltc, name, window):  # noqa: F811
    banner(f"long tiles {name} window {window}")
    H, G, D, page, codes, dtype, new, past = SHAPES[name]
    s = Setup(ltc, 101, H, D, page, codes, dtype, new, past)
    # the kernel's conditions: more packed rows a sequence than this, and this many workgroups
    assert s.rows * G // len(new) > 128 and (s.rows * G // 128 + len(new)) * H >= (512 if D <= 128 else 256)
    q, q64 = s.rows16(H * G, 2.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
    s.cache.check()
    assert bool(torch.isfinite(out).all())
    again = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
    assert torch.equal(out, again)
    scale = 2.0 ** (s.o["scales"].astype(np.float64) - 127)
    for i, length in enumerate(s.lengths):
        r0, r1 = int(s.cu[i]), int(s.cu[i + 1])
        if r0 == r1:
            continue
        pick = np.unique(np.concatenate([[r0, r1 - 1], s.rng.integers(r0, r1, 12)]))
        got = out[torch.from_numpy(pick).cuda()].double().cpu().numpy()
        pages = s.table[i, :-(-length // page)]
        position = length - (r1 - r0) + pick - r0
        t = np.arange(len(pages) * page)
        seen = t <= position[:, None]
        if window:
            seen &= t > position[:, None] - window
        for h in range(H):
            k, v = (np.nan_to_num(co.value(s.o[n][pages, h], codes)) * scale[pages, h, kind, None, None]
                    for kind, n in enumerate("kv"))
            k, v, vs = k.reshape(-1, D), v.reshape(-1, D), np.repeat(scale[pages, h, 1], page)
            for g in range(G):
                x = q64[pick, h * G + g]
                p = D ** -0.5 * (x @ k.T)
                big = D ** -0.5 * np.where(seen, np.abs(x) @ np.abs(k).T, 0).max(-1)
                p = np.where(seen, np.exp(p - np.where(seen, p, -np.inf).max(-1, keepdims=True)), 0)
                below = p.sum(-1, keepdims=True)
                want, mean, m = p @ v / below, p @ np.abs(v) / below, seen.sum(-1)
                # weights are off by 2^-11 of themselves, or 2^-34 of the largest times its scale; scores by dim + 8
                # roundings in 32 bits of the sum of magnitudes, twice, and 2^-22; sums by as many as positions, twice
                off = 2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -22 + 2 * m * 2.0 ** -24
                floor = m * 2.0 ** -34 * (p * vs).max(-1) / below[:, 0] * co.TOP[codes]
                slack = 1.01 * (off[:, None] * mean + floor[:, None])
                bad = np.abs(got[:, h * G + g] - want) > slack + HALF[dtype] * (np.abs(want) + slack) + SMALLEST[dtype]
                assert not bad.any(), (i, h, g, np.argwhere(bad)[:5])
