"""The 4-bit cache, weights, eviction and rotation without a GPU: arithmetic
that runs on the host too, and every argument error before anything is enqueued."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import cache4_oracle as c4
import evict_oracle as eo
from cache_cpu import GPU, cpu_cache, sequences
from lossless_tensor_compression_amd import LTCError
from lossless_tensor_compression_amd import kv_cache as kc
from lossless_tensor_compression_amd import rotation as rot
from test_cache_host import P, _lib, cache, rows, seqs

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "lossless_tensor_compression_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_host_arithmetic(tmp_path):
    exe = str(tmp_path / "cache4_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-I", CSRC, os.path.join(HERE, "cache4_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


# ---- the oracle against the definition and torch


def test_oracle_codes():
    """Ties, and the nearest of the sixteen for many numbers."""
    ties = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]
    assert [int(c4.code(x)) for x, _ in ties] == [c for _, c in ties]
    assert [int(c4.code(-x)) for x, _ in ties] == [c + 8 for _, c in ties]
    assert [int(c4.code(x)) for x in (np.inf, -np.inf, np.nan, -0.0, 7.0)] == [7, 15, 0, 8, 7]
    x = np.random.default_rng(0).uniform(-6, 6, 10000)
    grid = c4.value(np.arange(16, dtype=np.uint8))
    assert np.array_equal(np.abs(c4.value(c4.code(x)) - x), np.abs(grid[:, None] - x).min(0))


def test_oracle_layout_round_trip():
    rng = np.random.default_rng(1)
    for dim in kc.DIMS:
        shape = (3, 2, 32)
        c = {"k": rng.integers(0, 16, (*shape, dim)).astype(np.uint8), "v": rng.integers(0, 16, (*shape, dim)).astype(np.uint8),
             "ke": rng.integers(0, 256, shape).astype(np.uint8), "ve": rng.integers(0, 256, shape).astype(np.uint8),
             "drops": rng.integers(0, 16, (*shape, dim // 32)).astype(np.uint8)}
        stored = c4.to_stored(c)
        assert stored[0].shape == (3, 2, 2, dim // 32, 16, 16) and stored[1].shape == (3, 2, 2, dim, 8)
        assert stored[2].shape == (3, 2, 32 * (2 + kc.DROP_BYTES[dim]))
        again = c4.from_stored(*stored)
        assert all(np.array_equal(again[n], c[n]) for n in c)
        # by the document: token 19 of page 1, head 1, dims 37 and 38
        k = stored[0][1, 1, 1, 1, 3]
        assert (k[2] >> 4, k[3] & 15) == (c["k"][1, 1, 19, 37], c["k"][1, 1, 19, 38])
        assert stored[1][1, 1, 1, 37, 1] >> 4 == c["v"][1, 1, 19, 37]
        drops = stored[2][1, 1, 64 + 19 * kc.DROP_BYTES[dim]]
        assert (drops & 15, drops >> 4) == (c["drops"][1, 1, 19, 0], c["drops"][1, 1, 19, 1])


def test_oracle_pick():
    nan = float("nan")
    assert eo.pick(np.array([3.0, 1, 2, 3, nan, 0]), 3, 1) == [0, 3, 5]
    assert eo.pick(np.array([nan, nan, 1.0, nan]), 2, 0) == [0, 2]
    assert eo.pick(np.array([1.0, 1, 1, 1, 1]), 3, 1) == [0, 1, 4]
    assert eo.pick(np.array([1.0, 2, 3]), 3, 0) == eo.pick(np.array([1.0, 2, 3]), 9, 5) == [0, 1, 2]
    assert eo.pick(np.array([9.0, 2, 3]), 1, 1) == [2]


# ---- argument errors of the C ABI


def attend_weigh(c, s, x=None, q_heads=4, window=0, scale=0.1, out=P, weights=P, ws=P, ws_n=1 << 40):
    return _lib().ltc_cache_attend_weigh(ctypes.byref(c), s, rows() if x is None else x, q_heads, window, scale, out, weights, ws,
                                         ws_n, None)


def evict(c, s, weights=P, to=P, stride=4, width=4, keep=20, recent=4, lengths=P, positions=P, ws=P, ws_n=1 << 40):
    return _lib().ltc_cache_evict(ctypes.byref(c), s, weights, to, stride, width, keep, recent, lengths, positions, ws, ws_n, None)


def test_four_bit_caches_are_checked():
    L = _lib()
    for kw, code in ((dict(codes=2), -2), (dict(codes=4), -2), (dict(codes=3, s=P + 8), -1), (dict(codes=3, dim=80), -1),
                     (dict(codes=3, page=24), -1), (dict(codes=3, dtype=0), -2)):
        c = cache(**kw)
        assert L.ltc_cache_write(ctypes.byref(c), seqs(), rows(), rows(), None) == code
        assert L.ltc_cache_read(ctypes.byref(c), seqs(), P, P, None) == code
        assert L.ltc_cache_attend(ctypes.byref(c), seqs(), rows(), 4, 0, 0.1, P, P, 1 << 40, None) == code
        assert attend_weigh(c, seqs()) == code and evict(c, seqs(cu=0, n=3, rows=3)) == code
    assert L.ltc_cache_write(ctypes.byref(cache(codes=3)), seqs(n=0, rows=0), rows(base=0), rows(base=0), None) == 0


@pytest.mark.parametrize("codes", [0, 1, 3])
def test_weigh_refusals(codes):
    c = cache(codes=codes)
    for kw in (dict(q_heads=0), dict(q_heads=3), dict(window=1 << 31), dict(scale=0.0), dict(scale=float("nan")), dict(out=P + 2),
               dict(weights=0), dict(weights=P + 2), dict(x=rows(r=129))):
        assert attend_weigh(c, seqs(), **kw) == -1
    need = _lib().ltc_cache_attend_weigh_workspace_size(ctypes.byref(c), seqs(), 4, 0)
    assert need >= 65536 + 7 * 4 * 4
    for kw in (dict(ws=0), dict(ws=P + 4), dict(ws_n=need - 1)):
        assert attend_weigh(c, seqs(), **kw) == -7
    assert attend_weigh(c, seqs(rows=0), x=rows(base=0), weights=0, ws=0, ws_n=0) == 0  # nothing to do


def test_evict_refusals():
    c, s = cache(codes=3), seqs(cu=0, n=3, rows=3)
    for kw in (dict(keep=0), dict(recent=21), dict(width=1), dict(stride=3), dict(weights=0), dict(weights=P + 4), dict(to=0),
               dict(to=P + 2), dict(lengths=0), dict(positions=P + 1), dict(keep=65536 * 16 + 1, width=1 << 20, stride=1 << 20)):
        assert evict(c, s, **kw) == -1, kw
    assert evict(c, seqs()) == -1                             # row offsets have no meaning here
    assert evict(c, seqs(cu=0, n=65536, rows=65536)) == -1
    assert evict(c, seqs(cu=0, n=0, rows=0), weights=0, to=0, lengths=0, positions=0, ws=0, ws_n=0) == 0
    wide = seqs(cu=0, n=3, rows=3, width=4000, stride=4000)
    need = _lib().ltc_cache_evict_workspace_size(ctypes.byref(c), wide)
    assert need > 65536 and _lib().ltc_cache_evict_workspace_size(ctypes.byref(c), s) == 0
    for kw in (dict(ws=0), dict(ws=P + 4), dict(ws_n=need - 1)):
        assert evict(c, wide, **kw) == -7


def rotate(turns=P, status=P, dim=64, rotary=64, pairs=0, reserved=0, s=None, q=None, k=None, qw=P, kw=P, qo=P, ko=P, q_heads=2,
           k_heads=1, eps=1e-6, dtype=1):
    r = rot.RotationStruct(turns, status, dim, rotary, pairs, reserved)
    x = (rows() if q is None else q) + (rows() if k is None else k) + rot._pack_rest(qw, kw, qo, ko, q_heads, k_heads, eps, dtype)
    return _lib().ltc_norm_rotate(ctypes.byref(r), seqs(table=0) if s is None else s, x, None)


def test_rotate_refusals():
    assert ctypes.sizeof(rot.RotationStruct) == 32
    for kw in (dict(turns=0), dict(turns=P + 4), dict(status=0), dict(dim=80), dict(rotary=80), dict(rotary=24), dict(pairs=2),
               dict(reserved=1), dict(s=seqs(lengths=0)), dict(s=seqs(cu=P + 2)), dict(s=seqs(cu=0)), dict(s=seqs(n=0)),
               dict(s=seqs(rows=(1 << 24) + 1)), dict(s=seqs(reserved=1)), dict(q=rows(base=0)), dict(k=rows(r=12)),
               dict(qw=P + 2), dict(kw=P + 8), dict(qo=0), dict(ko=P + 4), dict(q_heads=65536), dict(k_heads=70000), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert rotate(**kw) == -1, kw
    assert rotate(dtype=0) == rotate(dtype=3) == -2
    assert rotate(s=seqs(n=0, rows=0)) == rotate(s=seqs(rows=0), q=rows(base=0)) == 0


# ---- the bindings


def test_layouts_that_do_not_fit(monkeypatch):
    """E2M1 tensors of the 8-bit layouts, and the other way round."""
    monkeypatch.setattr(kc, "lib", lambda: None)
    u8 = torch.uint8
    good = (torch.zeros(3, 2, 1, 2, 16, 16, dtype=u8), torch.zeros(3, 2, 1, 64, 8, dtype=u8), torch.zeros(3, 2, 16 * 3, dtype=u8))
    assert kc.KVCache._shape(*good, "e2m1") == (3, 2, 16, 64)
    eight = (torch.zeros(3, 2, 1, 4, 16, 16, dtype=u8), torch.zeros(3, 2, 1, 64, 16, dtype=u8), torch.zeros(3, 2, 2, dtype=u8))
    assert kc.KVCache._shape(*eight, "int8") == (3, 2, 16, 64)
    for i in range(3):
        mixed = [*good]
        mixed[i] = eight[i]
        with pytest.raises(ValueError):
            kc.KVCache._shape(*mixed, "e2m1")
        mixed = [*eight]
        mixed[i] = good[i]
        with pytest.raises(ValueError):
            kc.KVCache._shape(*mixed, "e4m3")


def binding(monkeypatch, **calls):
    c = cpu_cache(monkeypatch, **{"ltc_cache_attend": lambda *a: 0})
    for name, f in {"ltc_cache_attend_weigh": lambda *a: 0, "ltc_cache_attend_weigh_workspace_size": lambda *a: 0,
                    "ltc_cache_evict": lambda *a: 0, "ltc_cache_evict_workspace_size": lambda *a: 0, **calls}.items():
        setattr(c._lib, name, f)
    return c


def test_weights_that_are_refused(monkeypatch):
    reached = []
    c = binding(monkeypatch, ltc_cache_attend_weigh=lambda *a: reached.append(a) or 0, ltc_cache_evict=lambda *a: reached.append(a) or 0)
    q, (table, lengths), w = torch.zeros((1, 4, 64), dtype=torch.bfloat16), sequences([9]), torch.zeros((3, 2, 16))
    to = torch.zeros((1, 4), dtype=torch.int32)
    for bad in (w.double(), w[:2], w[..., :8], w.transpose(1, 2).contiguous().transpose(1, 2), w.clone().requires_grad_()):
        with pytest.raises(ValueError):
            kc.cache_attend(c, q, table, lengths, weights=bad)
        with pytest.raises(ValueError):
            kc.cache_evict(c, bad, table, lengths, to, 4)
    assert not reached
    kc.cache_attend(c, q, table, lengths, weights=w)
    kc.cache_evict(c, w, table, lengths, to, 4)
    assert len(reached) == 2


@pytest.mark.parametrize("keep,recent", [(0, 0), (-1, 0), (4, 5), (4, -1), (2 ** 32 + 4, 0), (4, 2 ** 32), (2 ** 31, 0)])
def test_budgets_that_are_refused(monkeypatch, keep, recent):
    reached = []
    c = binding(monkeypatch, ltc_cache_evict=lambda *a: reached.append(a) or 0)
    table, lengths = sequences([9])
    with pytest.raises(LTCError) as e:
        kc.cache_evict(c, torch.zeros((3, 2, 16)), table, lengths, torch.zeros((1, 4), dtype=torch.int32), keep, recent)
    assert e.value.code == -1 and not reached


def test_targets_that_are_refused(monkeypatch):
    c = binding(monkeypatch)
    table, lengths = sequences([9, 8])
    w, to = torch.zeros((3, 2, 16)), torch.zeros((2, 4), dtype=torch.int32)
    for bad in (to.long(), to[:1], to[:, :1], to.t().contiguous().t(), to[:1].expand(2, -1), to[0]):
        with pytest.raises(ValueError):
            kc.cache_evict(c, w, table, lengths, bad, 20)
    new, positions = kc.cache_evict(c, w, table, lengths, to, 20)
    assert new.shape == (2,) and positions.shape == (2, 2, 20) and positions.dtype == torch.int32


def test_turns():
    """Rates as 64-bit fractions of a turn, exact to the rate's own 2^-53."""
    for rate in (1.0, 0.1, 1e-9, 2 * math.pi, -1.0, 100.0):
        t, = rot.turns_of([rate])
        assert 0 <= t < 1 << 64
        x = rate / (2 * math.pi)
        assert abs((t / 2.0 ** 64 - x + 0.5) % 1.0 - 0.5) < 2.0 ** -50 * max(1.0, abs(x))
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            rot.turns_of([bad])


@pytest.mark.parametrize("kw", [dict(dim=80), dict(dim=64, rotary=65), dict(dim=64, rotary=24), dict(dim=64, rotary=80), dict(dim=64, rotary=-16),
                                dict(dim=64, theta=0.0), dict(dim=64, theta=float("nan")), dict(dim=64, rates=[1.0] * 31),
                                dict(dim=64, rates=[1.0] * 31 + [float("inf")])])
def test_rotations_that_are_refused(kw):
    with pytest.raises(ValueError):
        rot.Rotation(**kw, device="cpu")


def test_rotate_binding(monkeypatch):
    """What reaches the library, and what does not."""
    got = []
    monkeypatch.setattr(kc, "_current_gpu", lambda: GPU)
    monkeypatch.setattr(kc, "_raw_stream", lambda index: 0)
    import types
    monkeypatch.setattr(rot, "lib", lambda: types.SimpleNamespace(ltc_norm_rotate=lambda *a: got.append(a) or 0))
    r = rot.Rotation(64, device="cpu")
    q, k = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    lengths, w = torch.tensor([5, 6, 7], dtype=torch.int32), torch.ones(64, dtype=torch.bfloat16)
    leaf = q.clone().requires_grad_()
    for args, kw in (((q.float().half(), k), {}), ((q, k[:2]), {}), ((q[..., :32], k), {}), ((leaf, k), {}), ((leaf * 1, k), {}),
                     ((q, k), dict(q_weight=w.half())), ((q, k), dict(k_weight=w[:32])), ((q, k), dict(q_weight=w.clone().requires_grad_()))):
        with pytest.raises(ValueError):
            rot.norm_rotate(*args, r, lengths, **kw)
    for n, cu in ((lengths.long(), None), (lengths[:2], None), (lengths, lengths), (lengths.repeat(2)[::2], None)):
        with pytest.raises(ValueError):
            rot.norm_rotate(q, k, r, n, cu)
    with pytest.raises(LTCError):
        rot.norm_rotate(q.float(), k.float(), r, lengths)
    assert not got
    with torch.no_grad():
        a, b = rot.norm_rotate(leaf, k, r, lengths)
    assert a.shape == q.shape and b.shape == k.shape and not a.requires_grad and len(got) == 1 and len(got[0][2]) == 96
    strided = torch.zeros((3, 6, 64), dtype=torch.bfloat16)
    a, b = rot.norm_rotate(strided[:, :4], strided[:, 4:], r, lengths, q_weight=torch.ones(128, dtype=torch.bfloat16)[::2])
    assert a.is_contiguous() and b.is_contiguous()
