"""Queries and keys on their way to the cache: each head's norm and the
rotation by the row's position, in one pass.

  Rotation(dim, theta, rotary, pairs)            at which rates the dims turn
  norm_rotate(q, k, rotation, lengths, cu, q_weight, k_weight, eps)

A binding over ltc_norm_rotate of include/ltc.h.  Rows cu[i]..cu[i+1] belong to
sequence i and stand for its last positions, as in the cache's calls (see
kv_cache.py); lengths count the positions that a sequence has come to, which are
more than its cache holds once that has been cut.  Calls run on the current
stream, allocate nothing but their outputs and never synchronise.  They have no
backward pass: tensors that require a gradient are refused.
"""
import ctypes
import functools
import math
import struct

import torch

from . import LTCError, _check, lib
from . import kv_cache as _kc

_INT32 = torch.int32
_empty_like, _contiguous = torch.empty_like, torch.contiguous_format
_pack_rest = struct.Struct("=QQQQIIfi").pack  # ltc_rotate_rows behind its two ltc_cache_rows


class RotationStruct(ctypes.Structure):
    _fields_ = [("d_turns", ctypes.c_void_p), ("d_status", ctypes.c_void_p), ("dim", ctypes.c_uint32),
                ("rotary", ctypes.c_uint32), ("pairs", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


@functools.lru_cache(maxsize=None)
def _pi(bits):
    """pi * 2^bits, to the nearest few, by Machin's formula: 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan_of_inverse(n):
        total = term = (1 << (bits + 32)) // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    return (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


def turns_of(rates):
    """Angles of a position, in radians, as turns modulo 1 in 64 bits of
    fraction (Python integers), rounded down once: a quotient of doubles would be
    off by 2^-25 of a turn after 2^31 positions."""
    out = []
    for r in rates:
        if not math.isfinite(r):
            raise ValueError(f"rate {r}")
        n, d = float(r).as_integer_ratio()
        bits = 160 + (n.bit_length() + 63) // 64 * 64  # few different ones
        out.append((n << (63 + bits)) // (d * _pi(bits)) % (1 << 64))
    return out


class Rotation:
    """At which rates the first `rotary` of a head's dims turn (all of them by
    default): pair i by theta^(-2 i / rotary) radians a position, or by
    rates[i].  pairs: dims 2 i and 2 i + 1 are pair i; else dims i and
    i + rotary / 2."""

    def __init__(self, dim, theta=10000.0, rotary=None, pairs=False, rates=None, device="cuda"):
        rotary = dim if rotary is None else rotary
        if dim not in _kc.DIMS:
            raise ValueError(f"a head must have one of {_kc.DIMS} dims")
        if not 0 <= rotary <= dim or rotary % 16:
            raise ValueError("rotary must be a multiple of 16, up to dim")
        if rates is None:
            if not 0 < theta < math.inf:
                raise ValueError(f"theta {theta}")
            rates = [theta ** (-2.0 * i / rotary) for i in range(rotary // 2)]
        rates = [float(r) for r in rates]
        if len(rates) != rotary // 2:
            raise ValueError("rates must be [rotary / 2]")
        turns = [t - (1 << 64) if t >> 63 else t for t in turns_of(rates)]
        self.dim, self.rotary, self.pairs = dim, rotary, bool(pairs)
        self.turns = torch.tensor(turns, dtype=torch.int64, device=device)
        self.device = self.turns.device
        self.status = torch.zeros(1, dtype=_INT32, device=device)
        self._index, self._shape = self.turns.get_device(), torch.Size((dim,))
        self._lib = lib()
        self._struct = RotationStruct(self.turns.data_ptr(), self.status.data_ptr(), dim, rotary, int(self.pairs), 0)
        self._ref = ctypes.byref(self._struct)

    def check(self):
        """Raises if a call since the last check met lengths or cu that
        contradict each other (waits for the GPU)."""
        bits = int(self.status.item())
        self.status.zero_()
        if bits:
            raise LTCError(-5, "lengths or cu that contradict each other")


def _weight(t, rotation, dtype, name):
    """t in a form that the kernel takes (a copy where it is not)."""
    if t.dtype is not dtype or t.get_device() != rotation._index or t.shape != rotation._shape:
        raise ValueError(f"{name} must be {dtype} [{rotation.dim}] on the rotation's GPU")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which norm_rotate has not: call under torch.no_grad()")
    return t if t.stride(0) == 1 and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def norm_rotate(q, k, rotation, lengths, cu=None, q_weight=None, k_weight=None, eps=1e-6):
    """Queries [rows, q_heads, dim] and keys [rows, heads, dim] (bfloat16 or
    float16), each head x as x / sqrt(mean(x^2) + eps) * weight, turned by its
    row's position; without a weight it is turned alone.  Computed in 32 bits
    and rounded once.  Rows that belong to no sequence come out as zeros."""
    gpu = rotation._index
    if _kc._current_gpu() != gpu:
        if gpu < 0:
            raise ValueError("the rotation must be on a GPU")
        with torch.cuda.device(gpu):
            return norm_rotate(q, k, rotation, lengths, cu, q_weight, k_weight, eps)
    # straight code from here: it is most of a small call's time
    dtype = q.dtype
    if dtype not in _kc.CACHE_DTYPES:
        raise LTCError(-2, f"dtype {dtype}")
    if k.dtype is not dtype or q.get_device() != gpu or k.get_device() != gpu:
        raise ValueError("q and k must be of one type, on the rotation's GPU")
    q, qr, q_shape = _kc._take_rows(q, None, rotation.dim, "q")
    k, kr, k_shape = _kc._take_rows(k, None, rotation.dim, "k")
    rows = q_shape[0]
    if rows != k_shape[0]:
        raise ValueError("one key row for each query row")
    if not (lengths.dtype is _INT32 and lengths.get_device() == gpu
            and (cu is None or cu.dtype is _INT32 and cu.get_device() == gpu)):
        raise ValueError("lengths and cu must be int32 on the rotation's GPU")
    seqs = lengths.numel()
    if lengths.dim() != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous [sequences]")
    if cu is None:
        if rows != seqs:
            raise ValueError("without cu there is one row for each sequence")
    elif cu.dim() != 1 or cu.numel() != seqs + 1 or not cu.is_contiguous():
        raise ValueError("cu must be contiguous [sequences + 1]")
    if q_weight is not None:
        q_weight = _weight(q_weight, rotation, dtype, "q_weight")
    if k_weight is not None:
        k_weight = _weight(k_weight, rotation, dtype, "k_weight")
    # half the time of torch.empty with a shape
    q_out, k_out = _empty_like(q, memory_format=_contiguous), _empty_like(k, memory_format=_contiguous)
    s = _kc._pack_seqs(0, lengths.data_ptr(), 0 if cu is None else cu.data_ptr(), 0, seqs, rows, 0, 0)
    r = qr + kr + _pack_rest(0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(),
                             q_out.data_ptr(), k_out.data_ptr(), q_shape[1], k_shape[1], eps, _kc.CACHE_DTYPES[dtype])
    _check(rotation._lib.ltc_norm_rotate(rotation._ref, s, r, _kc._raw_stream(gpu)), "norm_rotate")
    return q_out, k_out
