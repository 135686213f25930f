"""Queries with infinities: the row's outputs are NaN, whatever the signs of
the keys; other rows, and rows that see nothing, are as ever."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, Setup, close, ltc  # noqa: F401
from test_gpu_cache_tiles import setup

pytestmark = pytest.mark.gpu


def check(ltc, s, q_heads, value, window=0):  # noqa: F811
    """Infinities in one dim of a key head of which every key is positive,
    so that the scores of -inf are all -inf."""
    dim = 9
    s.o["k"][..., dim] = 5
    s.upload(ltc)
    q, q64 = s.rows16(q_heads, 1.0)
    for row, head in ((0, 0), (s.rows - 1, q_heads - 1), (s.rows // 2, 1)):
        q[row, head, dim] = value
        q64[row, head, dim] = value
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
    with np.errstate(invalid="ignore"):
        want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu, window)
    assert 0 < np.isnan(want).sum() <= 3 * s.D
    close(out, want, np.where(np.isnan(slack), 0.0, slack), s.dtype)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("codes,dtype,dim", [("e4m3", BF, 128), ("int8", FP, 64), ("e4m3", FP, 96), ("int8", BF, 256)])
@pytest.mark.parametrize("new,past", [([1, 1, 1], [0, 80, 700]), ([1, 20], [0, 300]), ([40], [0])])
def test_rows(ltc, codes, dtype, dim, value, new, past):  # noqa: F811
    banner(f"query with {value}, {codes} {dim}, {new} after {past}")
    s = Setup(ltc, 95, 2, dim, 32, codes, dtype, new, past, single=max(new) == 1)
    check(ltc, s, 4, value)
    check(ltc, s, 4, value, window=3)


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["64 int8", "128"])
def test_tiles(ltc, name, value):  # noqa: F811
    banner(f"query with {value}, tiles {name}")
    s, q_heads = setup(ltc, name, 96)
    check(ltc, s, q_heads, value)


def test_nothing_seen(ltc):  # noqa: F811
    """Pages that are not there are not seen: zeros, not NaN."""
    s = Setup(ltc, 97, 2, 64, 16, "e4m3", BF, [1, 1], [0, 4], single=True)
    s.table[0, 0] = -1
    s.upload(ltc)
    q, q64 = s.rows16(4, 1.0)
    q[:, 1, 3], q64[:, 1, 3] = -float("inf"), -float("inf")
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, None)
    with np.errstate(invalid="ignore"):
        want, slack, bits = co.attend(s.o, q64, s.table, s.lengths)
    assert bits == 1 and not want[0].any()
    close(out, want, np.where(np.isnan(slack), 0.0, slack), BF)
