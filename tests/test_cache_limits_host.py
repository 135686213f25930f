"""Calls of the key/value cache that pass a grid's limits are refused on the
host; none of these needs a GPU."""
import ctypes

import pytest

from test_cache_host import P, _lib, cache, rows, seqs


@pytest.mark.parametrize("kw", [dict(n=(1 << 20) + 1, rows=5), dict(rows=(1 << 24) + 1)])
def test_rows_and_sequences(kw):
    L, c, s = _lib(), cache(), seqs(**kw)
    assert L.ltc_cache_write(ctypes.byref(c), s, rows(), rows(), None) == -1
    assert L.ltc_cache_read(ctypes.byref(c), s, P, P, None) == -1
    assert L.ltc_cache_attend(ctypes.byref(c), s, rows(), 4, 0, 0.1, P, P, 1 << 40, None) == -1
    assert L.ltc_cache_attend_workspace_size(ctypes.byref(c), s, 4, 0) == 0


@pytest.mark.parametrize("n,r,heads", [(3, 1 << 24, 128), (1 << 20, 1 << 20, 1026), (1, 1 << 16, 32768)])
def test_rows_times_heads(n, r, heads):
    """(rows + sequences) * query heads just past 2^31; one head fewer is only
    refused for its workspace."""
    L, c = _lib(), cache()
    s = seqs(n=n, rows=r)
    assert (n + r) * heads > 1 << 31
    assert L.ltc_cache_attend(ctypes.byref(c), s, rows(), heads, 0, 0.1, P, P, 1 << 40, None) == -1
    assert L.ltc_cache_attend_workspace_size(ctypes.byref(c), s, heads, 0) == 0


def test_too_small_a_workspace():
    L, c, s = _lib(), cache(), seqs(width=4000, stride=4000)
    need = L.ltc_cache_attend_workspace_size(ctypes.byref(c), s, 4, 0)
    assert need > 65536
    for ws, n in ((P, need - 1), (P + 128, need), (0, need)):
        assert L.ltc_cache_attend(ctypes.byref(c), s, rows(), 4, 0, 0.1, P, ws, n, None) == -7
