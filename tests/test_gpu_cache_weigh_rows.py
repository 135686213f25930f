"""Positions' weights where scores are not written down: few rows over wide
tables, and middling numbers of rows, of each code type and size of a head.
Which way a call takes is asked of its workspace, so that a later rule cannot
take these tests elsewhere unseen."""
import numpy as np
import pytest
import torch

import evict_oracle as eo
from cache4_setup import close
from gpu_util import banner
from test_gpu_cache_weigh import BF, FP, setup

pytestmark = pytest.mark.gpu

TYPES = [("e4m3", BF), ("int8", FP), ("e2m1", BF), ("e4m3", FP), ("int8", BF), ("e2m1", FP)]


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def widen(s, width):
    """More columns of the table, behind every sequence's end: anything."""
    table = s.rng.integers(-5, 2 ** 31 - 1, (len(s.lengths), width)).astype(np.int32)
    table[:, :s.table.shape[1]] = s.table
    s.table, s.gtable = table, torch.from_numpy(table).cuda()


def way(s, q_heads, window):
    """(scores are written down, the rows of a step are shared out over a workgroup's waves)"""
    lib, seqs = s.cache._lib, s.cache._seqs(s.gtable, s.glengths, s.gcu, s.rows)
    plain = max(lib.ltc_cache_attend_workspace_size(s.cache._ref, seqs, q_heads, window), 65536)
    more = lib.ltc_cache_attend_weigh_workspace_size(s.cache._ref, seqs, q_heads, window) - plain
    assert more >= s.rows * q_heads * 4
    mean = -(-s.rows * (q_heads // s.H) // len(s.lengths))
    steps = len(s.lengths) * s.H * -(-s.table.shape[1] * s.P // 64)
    return more > s.rows * q_heads * 4 + 1024, mean > 256 or (mean > 16 and steps < 4096)


def check(ltc, s, q_heads, window=0, calls=2):
    weights = torch.from_numpy(s.rng.exponential(1.0, tuple(s.cache.no_weights().shape)).astype(np.float32)).cuda()
    want_w, total = weights.double().cpu().numpy(), 0.0
    for _ in range(calls):
        q, q64 = s.rows16(q_heads, 2.0)
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, weights=weights)
        want, slack, shares, off, status = eo.attend(s.o, q64, s.table, s.lengths, s.cu, window)
        close(out, want, slack, s.dtype)
        want_w, slack_w = eo.weigh(s.o, want_w, shares, off, s.table, s.lengths, s.cu, s.rows)
        total = total + slack_w
        got = weights.double().cpu().numpy()
        bad = np.abs(got - want_w) > total
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want_w[bad][:5], total[bad][:5])
    assert int(s.cache.status.item()) == status
    return status


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("codes,dtype", TYPES)
def test_single_rows_of_wide_tables(ltc, codes, dtype, dim):
    """A wave's steps lie 512 positions apart: the long sequences have three of them."""
    banner(f"weigh single rows of wide tables, {codes}, dim {dim}")
    past = [(i * 7) % 40 for i in range(96)]
    past[5], past[31], past[64], past[95] = 1500, 511, 512, 1087
    s = setup(ltc, 111, 8, dim, 16, codes, dtype, [1] * 96, past, single=True)
    widen(s, 1500)
    assert way(s, 16, 0) == (False, False)
    assert check(ltc, s, 16) == 0


# with a narrower window the scores of 256 dims are written down
DRAFTS = [("e4m3", BF, 64), ("int8", FP, 96), ("e2m1", BF, 128), ("e4m3", FP, 192), ("int8", BF, 128), ("e2m1", FP, 64), ("e2m1", FP, 192),
          ("e2m1", BF, 256), ("int8", FP, 256), ("e4m3", BF, 256)]


@pytest.mark.parametrize("codes,dtype,dim,window", [(*d, w) for d in DRAFTS for w in ((0, 70, 1000) if d[2] < 256 else (0, 20000))])
def test_drafts(ltc, codes, dtype, dim, window):
    """Some rows a sequence, of an odd number of query heads: a wave's steps lie 1,024 positions apart."""
    banner(f"weigh drafts, {codes}, dim {dim}, window {window}")
    new = [3 + (i * 5) % 9 for i in range(48)]
    past = [(i * 11) % 90 for i in range(48)]
    past[0], past[20], past[47] = 1490, 1015, 1020
    s = setup(ltc, 112, 8, dim, 16, codes, dtype, new, past)
    widen(s, 3000)
    assert way(s, 24, window) == (False, False)
    assert check(ltc, s, 24, window, calls=1) == 0


@pytest.mark.parametrize("codes,dtype", TYPES[:3])
def test_bad_pages(ltc, codes, dtype):
    """Missing pages in the middle and at the end of both kinds of calls."""
    for new, single, width, q_heads in (([1] * 96, True, 1500, 16), ([3 + (i * 5) % 9 for i in range(48)], False, 1000, 24)):
        past = [(i * 7) % 60 + 40 for i in range(len(new))]
        past[5], past[31] = 1500, 1100
        s = setup(ltc, 113, 8, 64, 16, codes, dtype, new, past, single=single)
        for i in range(0, len(new), 3):
            s.table[i, (i * 5) % (s.lengths[i] // 16 + 1)] = -1 - i
        s.table[5, 63:67] = 2 ** 31 - 1
        widen(s, width)
        assert way(s, q_heads, 0) == (False, False)
        assert check(ltc, s, q_heads, calls=1) == 1


@pytest.mark.parametrize("codes,dtype", TYPES)
def test_large_heads_whose_rows_are_shared(ltc, codes, dtype):
    """256 dims, rows enough for a workgroup's waves to share them, a table too wide for scores."""
    s = setup(ltc, 114, 1, 256, 256, codes, dtype, [40], [500])
    widen(s, 800)
    assert way(s, 8, 0) == (False, True)
    assert check(ltc, s, 8) == 0
    s = setup(ltc, 115, 1, 256, 16, codes, dtype, [40, 3, 90], [500, 70, 5])
    widen(s, 3500)
    assert way(s, 16, 0) == (False, True)
    assert check(ltc, s, 16, calls=1) == 0
