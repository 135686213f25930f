"""Rows of a call that belong to no sequence, before cu[0] and from cu[-1] on:
zeros in every output, and no part in what is written."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, Setup, close, ltc, same_cache  # noqa: F401
from test_gpu_cache_tiles import setup

pytestmark = pytest.mark.gpu


@pytest.fixture
def sevens(monkeypatch):
    """Outputs are made of memory that holds sevens."""
    empty, like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).fill_(7))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **kw: like(*a, **kw).fill_(7))


def widen(s, before, behind):
    """The call with rows of no sequence around its own; those of the rows
    that are given hold NaN."""
    s.cu = s.cu + np.int32(before)
    s.gcu = torch.from_numpy(s.cu).cuda()
    own, s.rows = s.rows, s.rows + before + behind

    def rows16(heads, size=1.0):
        x, x64 = Setup.rows16(s, heads, size)
        for y in (x, x64):
            y[:before], y[before + own:] = float("nan"), float("nan")
        return x, x64

    s.rows16 = rows16


CALLS = {
    "split": (2, 64, 16, "e4m3", BF, [1, 0, 3], [300, 20, 70]),
    "ragged": (5, 96, 32, "int8", FP, [15, 16, 1, 33, 47], [1, 0, 15, 16, 2]),
    "unsplit": (3, 128, 64, "e4m3", FP, [2] * 180, [(i * 7) % 90 for i in range(180)]),
    "no rows at all": (2, 256, 64, "int8", BF, [0, 0], [5, 0]),
    "two waves": (8, 256, 16, "e4m3", BF, [9] * 40, [(i * 5) % 50 for i in range(40)]),
}


@pytest.mark.parametrize("before,behind", [(3, 0), (0, 1), (200, 517)])
@pytest.mark.parametrize("call", list(CALLS))
def test_rows(ltc, sevens, call, before, behind):  # noqa: F811
    banner(f"unnamed rows {call} {before} {behind}")
    s = Setup(ltc, 91, *CALLS[call])
    widen(s, before, behind)
    q, q64 = s.rows16(s.H * 3, 2.0)
    for window in (0, 10):
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
        want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu, window)
        close(out, want, slack, s.dtype)
    for got, want in zip(ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows),
                         co.read(s.o, s.table, s.lengths, s.cu, s.rows)):
        close(got, want, 0.0, s.dtype)
    k, k64 = s.rows16(s.H)
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    s.o, _ = co.write(s.o, k64, k64, s.table, s.lengths, s.cu)
    same_cache(s, s.o)
    s.cache.check()


@pytest.mark.parametrize("name", ["64", "128 odd", "256"])
def test_tiles(ltc, sevens, name):  # noqa: F811
    banner(f"unnamed rows, tiles {name}")
    s, q_heads = setup(ltc, name, 92)
    widen(s, 150, 70)
    q, q64 = s.rows16(q_heads, 2.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, s.dtype)
    s.cache.check()


def test_fewer_rows_in_a_graph(ltc):  # noqa: F811
    """A captured call whose row offsets change between replays."""
    s = Setup(ltc, 93, 2, 64, 16, "e4m3", BF, [4, 4, 4], [30, 9, 100])
    q, q64 = s.rows16(4, 2.0)
    step = lambda: (ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu),  # noqa: E731
                    *ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=12))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for cu in ([0, 4, 8, 12], [0, 4, 4, 6], [2, 3, 5, 9], [0, 0, 0, 0], [12, 12, 12, 12], [0, 4, 8, 12]):
        s.cu = np.array(cu, np.int32)
        s.gcu.copy_(torch.from_numpy(s.cu))
        for x in held:
            x.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu)
        close(held[0], want, slack, BF)
        for got, want in zip(held[1:], co.read(s.o, s.table, s.lengths, s.cu, 12)):
            close(got, want, 0.0, BF)
    s.cache.check()
