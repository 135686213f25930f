"""What no row of a call sees has no part in its bits: exponents behind the
sequences' ends, those of the cache's first page, which is read in their place,
and those before the windows."""
import numpy as np
import pytest
import torch

from cache4_setup import Setup4
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def bits(ltc, s, q, window):
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
    return out.view(torch.int16).clone()


@pytest.mark.parametrize("dim,dtype,heads,group,new,past", [(128, BF, 2, 4, [1, 5, 1], [200, 300, 77]), (64, FP, 1, 3, [40, 3], [70, 333]),
                                                            (256, BF, 2, 2, [1, 1], [900, 30]),
                                                            (128, BF, 8, 16, [7 + i % 5 for i in range(64)], [(i * 29) % 130 for i in range(64)]),
                                                            (64, FP, 8, 16, [7 + i % 5 for i in range(64)], [(i * 29) % 130 for i in range(64)])])
@pytest.mark.parametrize("window", [0, 50])
def test_unseen_exponents(ltc, dim, dtype, heads, group, new, past, window):
    banner(f"unseen exponents, dim {dim}, window {window}")
    s = Setup4(ltc, 141, heads, dim, 16, dtype, new, past)
    # the cache's first page is no sequence's
    free = int(s.free[0])
    swap = {0: free, free: 0}
    s.table = np.vectorize(lambda p: swap.get(int(p), int(p)))(s.table).astype(np.int32)
    for name in s.o:
        s.o[name][[0, free]] = s.o[name][[free, 0]]
    s.upload(ltc)
    seen = np.zeros(s.o["ve"].shape, bool)
    for i, (n, p) in enumerate(zip(new, past)):
        for t in range(max(p + 1 - window, 0) if window else 0, n + p):
            seen[s.table[i, t // 16], :, t % 16] = True
    q, _ = s.rows16(heads * group, 1.0)
    s.o["ve"][~seen] = 127
    s.upload(ltc)
    want = bits(ltc, s, q, window)
    for low, high in ((27, 28), (253, 254), (0, 256)):
        for name in ("ke", "ve"):
            s.o[name][~seen] = s.rng.integers(low, high, int((~seen).sum()))
        s.upload(ltc)
        assert torch.equal(bits(ltc, s, q, window), want)
