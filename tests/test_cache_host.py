"""Host-side checks of the key/value cache's C ABI that need no GPU: every
argument error is returned before anything is enqueued."""
import ctypes
import os

import pytest

ltc = pytest.importorskip("lossless_tensor_compression_amd")
from lossless_tensor_compression_amd import kv_cache as kc  # noqa: E402

P = 1 << 20  # stands for a device pointer; never followed on the host


def _lib():
    if not os.path.exists(ltc.LIB_PATH):
        import lossless_tensor_compression_amd.build as b
        b.build()
    return ltc.lib()


def cache(**kw):
    d = dict(k=P, v=P, s=P, status=P, pages=10, heads=2, dim=64, page=16, codes=0, dtype=1)
    d.update(kw)
    return kc.CacheStruct(*d.values())


def seqs(table=P, lengths=P, cu=P, stride=4, n=3, rows=7, width=4, reserved=0):
    return kc._pack_seqs(table, lengths, cu, stride, n, rows, width, reserved)


def rows(base=P, r=128, h=64):
    return kc._pack_rows(base, r, h)


def calls(c, s, x=None, q_heads=4, window=0, scale=0.1, out=P, ws=P, ws_n=1 << 40):
    L, c = _lib(), ctypes.byref(c) if c is not None else None
    x = rows() if x is None else x
    return (L.ltc_cache_write(c, s, x, x, None), L.ltc_cache_read(c, s, out, out, None),
            L.ltc_cache_attend(c, s, x, q_heads, window, scale, out, ws, ws_n, None))


def test_struct_sizes():
    assert ctypes.sizeof(kc.CacheStruct) == 56 and len(seqs()) == 48 and len(rows()) == 24


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -2), (dict(dtype=3), -2), (dict(codes=2), -2), (dict(codes=-1), -2),
    (dict(page=0), -1), (dict(page=8), -1), (dict(page=48), -1), (dict(page=512), -1),
    (dict(dim=0), -1), (dict(dim=80), -1), (dict(dim=512), -1), (dict(heads=0), -1), (dict(heads=70000), -1),
    (dict(pages=(1 << 30) + 1), -1), (dict(k=0), -1), (dict(v=P + 8), -1), (dict(s=P + 1), -1), (dict(status=0), -1)])
def test_cache_refusals(kw, code):
    assert calls(cache(**kw), seqs()) == (code,) * 3


@pytest.mark.parametrize("kw", [
    dict(table=0), dict(lengths=0), dict(lengths=P + 2), dict(cu=P + 1), dict(cu=0), dict(stride=3),
    dict(n=0), dict(rows=(1 << 24) + 1), dict(n=(1 << 22) + 1), dict(reserved=1)])
def test_sequence_refusals(kw):
    assert calls(cache(), seqs(**kw)) == (-1,) * 3


def test_row_refusals():
    for x in (rows(base=0), rows(base=P + 8), rows(r=129), rows(h=4)):
        w, _, a = calls(cache(), seqs(), x, out=P + 2)
        assert w == -1 and a == -1
    L, c = _lib(), cache()
    assert L.ltc_cache_read(ctypes.byref(c), seqs(), P + 4, P, None) == -1
    for kw in (dict(q_heads=0), dict(q_heads=3), dict(q_heads=65538), dict(window=1 << 31), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=P + 2)):
        d = dict(q_heads=4, window=0, scale=0.1, out=P)
        d.update(kw)
        assert L.ltc_cache_attend(ctypes.byref(c), seqs(), rows(), d["q_heads"], d["window"], d["scale"], d["out"],
                                  P, 1 << 40, None) == -1
    assert L.ltc_cache_write(None, seqs(), rows(), rows(), None) == -1
    assert L.ltc_cache_write(ctypes.byref(c), None, rows(), rows(), None) == -1
    assert L.ltc_cache_write(ctypes.byref(c), seqs(), None, rows(), None) == -1


def test_nothing_to_do_needs_no_gpu():
    empty = seqs(n=0, rows=0)
    assert calls(cache(pages=0, k=0, v=0, s=0), empty, rows(base=0)) == (0, 0, 0)
    assert calls(cache(), seqs(rows=0), rows(base=0)) == (0, 0, 0)
