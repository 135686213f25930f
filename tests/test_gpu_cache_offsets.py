"""Row offsets that contradict each other: always reported; where they only
leave the call's rows, all other sequences are served; nothing of a refused
sequence is written."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, Setup, close, ltc, same_cache  # noqa: F401
from test_gpu_cache_tiles import setup

pytestmark = pytest.mark.gpu


def status(s):
    bits = int(s.cache.status.item())
    s.cache.status.zero_()
    return bits


@pytest.mark.parametrize("cu", [[0, 20, 25, 58, 63], [-1, 20, 25, 58, 62], [0, 20, 25, 58, 2 ** 31 - 1],
                                [-2 ** 31, 20, 25, 58, 62], [0, 20, 25, 25, 25]])
@pytest.mark.parametrize("codes,dtype", [("int8", FP), ("e4m3", BF)])
def test_others_are_served(ltc, codes, dtype, cu):  # noqa: F811
    """Offsets that leave the rows, or (the last) a sequence of fewer
    positions than rows beside one without rows."""
    banner(f"offsets {cu} {codes}")
    s = Setup(ltc, 42, 2, 64, 16, codes, dtype, [20, 5, 33, 4], [30, 0, 40, 9])
    if cu[2:4] == [25, 25]:
        s.lengths[0] = 19
    s.cu = np.array(cu, np.int32)
    s.upload(ltc)
    q, q64 = s.rows16(6, 2.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, bits = co.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, dtype)
    assert status(s) == bits == 2
    for got, want in zip(ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows),
                         co.read(s.o, s.table, s.lengths, s.cu, s.rows)):
        close(got, want, 0.0, dtype)
    assert status(s) == 2
    k, k64 = s.rows16(2)
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    s.o, bits = co.write(s.o, k64, k64, s.table, s.lengths, s.cu)
    same_cache(s, s.o)
    assert status(s) == bits == 2


@pytest.mark.parametrize("cu", [[0, 33, 38, 10, 75], [0, 32, 35, 25, 63], [0, 2 ** 31 - 1, 25, -2 ** 31, 62],
                                [0, 17, 21, 39, 51, 75, 92, 49, 127, 142], [0, 29, 66, 96, 123, 124, 129, 148, 134, 202],
                                [0, 9, 10, 11, 22, 33, 109, 69, 102, 118]])
def test_decreasing(ltc, cu):  # noqa: F811
    """Among them offsets whose sequence at fault no workgroup finds by its
    search."""
    banner(f"decreasing offsets {cu}")
    n = len(cu) - 1
    s = Setup(ltc, 43, 2, 64, 16, "e4m3", BF, [0] * n, [400] * n, nan_behind=False)
    s.cu = np.array(cu, np.int32)
    s.rows = cu[-1]
    s.upload(ltc)
    before = [x.copy() for x in s.got()]
    k, _ = s.rows16(2)
    for q_heads in (2, 4, 32):
        q, _ = s.rows16(q_heads)
        for window in (0, 30):
            ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
            assert status(s) == 2
    ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
    assert status(s) == 2
    for a, b in zip(before, s.got()):
        assert np.array_equal(a, b)
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    assert status(s) == 2
    served = [p for i, (_, _, _, ok) in enumerate(co.spans(s.cu, s.lengths, s.rows, s.table.shape[1] * 16)) if ok
              for p in s.table[i, :25]]
    rest = np.setdiff1d(np.arange(len(before[2])), served)
    assert len(rest) >= 27  # a refused sequence's pages and two of none
    for a, b in zip(before, s.got()):
        assert np.array_equal(a[rest], b[rest])


def test_decreasing_tiles(ltc):  # noqa: F811
    banner("decreasing offsets, tiles")
    s, q_heads = setup(ltc, "64", 94)
    assert len(s.cu) == 25
    cu = [0, 6, 13, 24, 36, 47, 58, 50, 72, 77, 81, 85, 95, 105, 110, 116, 127, 133, 139, 145, 150, 162, 170, 182, 187]
    gcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lengths = torch.full((24,), 100, dtype=torch.int32, device="cuda")
    table = torch.zeros((24, 8), dtype=torch.int32, device="cuda")
    q = torch.ones((187, q_heads, 64), dtype=BF, device="cuda")
    assert (187 * 16 // 128 + 24) * 16 >= 512
    ltc.cache_attend(s.cache, q, table, lengths, gcu)
    assert status(s) == 2
