"""A paged key/value cache in 8 bits: quantised as it is written, read back,
and attended to in place.

  KVCache.empty(...) / KVCache.of(...)  the cache's tensors and their layout
  cache_write(cache, k, v, table, lengths, cu)   new keys and values to their positions
  cache_read(cache, table, lengths, cu, rows)    positions back as 16-bit rows
  cache_attend(cache, q, table, lengths, cu)     attention of new queries

A binding over ltc_cache_write, ltc_cache_read and ltc_cache_attend of
include/ltc.h, where the layouts, the rounding and what happens with bad
tables are written down.  Calls run on the current stream, allocate nothing
but their outputs and a workspace that the cache keeps for each stream, and
never synchronise, so they can be captured in a graph.  They have no backward
pass: rows that require a gradient are refused.  Threads may share a
cache; their calls on one stream run in the order in which they are made.

Rows cu[i]..cu[i+1] of a call belong to sequence i and stand for its last
positions, lengths[i] - (cu[i+1] - cu[i]) to lengths[i] - 1; without cu each
sequence has one row.  Rows outside cu[0]..cu[-1] belong to no sequence and
come out as zeros.  Position t of sequence i is token t % page of page
table[i, t // page].  table, lengths and cu are int32 tensors on the GPU.
"""
import ctypes
import struct
import threading

import torch

from . import LTCError, _check, lib

E4M3, INT8 = 0, 1
CODES = {"e4m3": E4M3, "int8": INT8}
CACHE_DTYPES = {torch.bfloat16: 1, torch.float16: 2}
PAGES = (16, 32, 64, 128, 256)
DIMS = (64, 96, 128, 192, 256)
BAD_PAGE, BAD_SEQUENCE = 1, 2
WS_ZEROS = 65536

_INT32 = torch.int32
_current_gpu = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() builds a Stream object: 2.7 us a call
_pack_seqs = struct.Struct("=QQQQIIII").pack      # ltc_cache_seqs
_pack_rows = struct.Struct("=QQQ").pack           # ltc_cache_rows


class CacheStruct(ctypes.Structure):
    _fields_ = [("d_k_codes", ctypes.c_void_p), ("d_v_codes", ctypes.c_void_p), ("d_scales", ctypes.c_void_p),
                ("d_status", ctypes.c_void_p), ("pages", ctypes.c_uint32), ("heads", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("page", ctypes.c_uint32), ("codes", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class KVCache:
    """The tensors of a cache and what the library has to know of them.

    k_codes uint8 [pages, heads, page/16, dim/16, 16 tokens, 16 dims]
    v_codes uint8 [pages, heads, page/16, dim, 16 tokens]
    scales  uint8 [pages, heads, 2], a scale is 2^(byte - 127)
    dtype: torch.bfloat16 or torch.float16, of keys, values, queries and
    outputs; codes: "e4m3" or "int8"."""

    def __init__(self, k_codes, v_codes, scales, dtype, codes):
        if codes not in CODES:
            raise LTCError(-2, f"codes {codes!r}")
        if dtype not in CACHE_DTYPES:
            raise LTCError(-2, f"dtype {dtype}")
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes), ("scales", scales)):
            if not t.is_cuda or t.device != k_codes.device:
                raise ValueError(f"{name} must be on the cache's GPU")
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous uint8")
        pages, heads, page, dim = self._shape(k_codes, v_codes, scales)
        self.k_codes, self.v_codes, self.scales = k_codes, v_codes, scales
        self.pages, self.heads, self.page, self.dim = pages, heads, page, dim
        self.dtype, self.codes, self.device = dtype, codes, k_codes.device
        self.status = torch.zeros(1, dtype=torch.int32, device=k_codes.device)
        self._lib = lib()
        self._struct = CacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), scales.data_ptr(), self.status.data_ptr(),
                                   pages, heads, dim, page, CODES[codes], CACHE_DTYPES[dtype])
        self._ref = ctypes.byref(self._struct)
        self._index = self.device.index
        self._workspaces = {}  # stream -> tensor, its first bytes zero between calls
        self._lock = threading.Lock()  # from a workspace's lookup to the launch that uses it

    @staticmethod
    def _shape(k_codes, v_codes, scales):
        if k_codes.dim() != 6 or k_codes.shape[4:] != (16, 16):
            raise ValueError("k_codes must be [pages, heads, page/16, dim/16, 16, 16]")
        pages, heads, blocks, parts = k_codes.shape[:4]
        if v_codes.shape != (pages, heads, blocks, parts * 16, 16):
            raise ValueError("v_codes must be [pages, heads, page/16, dim, 16]")
        if scales.shape != (pages, heads, 2):
            raise ValueError("scales must be [pages, heads, 2]")
        if blocks * 16 not in PAGES:
            raise ValueError(f"a page must have one of {PAGES} tokens")
        if parts * 16 not in DIMS:
            raise ValueError(f"a head must have one of {DIMS} dims")
        if heads < 1:
            raise ValueError("at least one head")
        return pages, heads, blocks * 16, parts * 16

    @classmethod
    def of(cls, k_codes, v_codes, scales, dtype=torch.bfloat16, codes="e4m3"):
        """A cache over tensors that the caller holds."""
        return cls(k_codes, v_codes, scales, dtype, codes)

    @classmethod
    def empty(cls, pages, heads, dim, page=64, dtype=torch.bfloat16, codes="e4m3", device="cuda"):
        """A cache with tensors of its own, zeros with the lowest scale."""
        if page not in PAGES or dim not in DIMS:
            raise ValueError(f"page must be one of {PAGES} and dim one of {DIMS}")
        return cls(torch.zeros((pages, heads, page // 16, dim // 16, 16, 16), dtype=torch.uint8, device=device),
                   torch.zeros((pages, heads, page // 16, dim, 16), dtype=torch.uint8, device=device),
                   torch.full((pages, heads, 2), 27, dtype=torch.uint8, device=device), dtype, codes)

    def check(self):
        """Raises if a call since the last check met a bad page or sequence
        (waits for the GPU)."""
        bits = int(self.status.item())
        self.status.zero_()
        if bits:
            what = [n for b, n in ((BAD_PAGE, "a table entry outside the cache"),
                                   (BAD_SEQUENCE, "lengths or cu that contradict each other")) if bits & b]
            raise LTCError(-5, " and ".join(what))

    def _workspace(self, need, stream):
        """A workspace for a call on the stream, for the caller to hold until
        it has launched.  Each stream keeps one, since its calls run in order;
        a captured call gets its own, which lives and is cleared with the
        graph."""
        captured = torch._C._cuda_isCurrentStreamCapturing()
        ws = None if captured else self._workspaces.get(stream)
        if ws is None or ws.numel() < need:
            ws = torch.empty(1 << (need - 1).bit_length(), dtype=torch.uint8, device=self.device)
            ws[:WS_ZEROS].zero_()
            if not captured:
                self._workspaces[stream] = ws
        return ws

    def _seqs(self, table, lengths, cu, rows):
        """ltc_cache_seqs as bytes; what can be seen without the GPU is checked.
        Straight code: it is half of a small call's time."""
        gpu = self._index
        if not (table.dtype is _INT32 and lengths.dtype is _INT32 and table.get_device() == gpu
                and lengths.get_device() == gpu and (cu is None or cu.dtype is _INT32 and cu.get_device() == gpu)):
            raise ValueError("table, lengths and cu must be int32 on the cache's GPU")
        shape, stride = table.shape, table.stride()
        seqs = lengths.numel()
        if len(shape) != 2 or shape[0] != seqs or lengths.dim() != 1:
            raise ValueError("table must be [sequences, pages] and lengths [sequences]")
        width = shape[1]
        if not lengths.is_contiguous() or (stride[1] != 1 and width > 1):
            raise ValueError("lengths and the rows of table must be contiguous")
        if cu is None:
            if rows != seqs:
                raise ValueError("without cu there is one row for each sequence")
        elif cu.dim() != 1 or cu.numel() != seqs + 1 or not cu.is_contiguous():
            raise ValueError("cu must be contiguous [sequences + 1]")
        step = stride[0] if seqs > 1 else width
        if step < width:
            raise ValueError("the rows of table must not overlap")
        return _pack_seqs(table.data_ptr(), lengths.data_ptr(), 0 if cu is None else cu.data_ptr(), step,
                          seqs, rows, width, 0)

    def _rows(self, t, heads, name):
        """t as rows that the kernels can take (a copy where its strides or
        alignment do not let them), its ltc_cache_rows as bytes and its shape."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name} must be {self.dtype} on the cache's GPU")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, which the cache's operators have not: call under torch.no_grad()")
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.dim or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be [rows, {'heads' if heads is None else heads}, {self.dim}]")
        r, h, d = t.stride()
        at = t.data_ptr()
        if d != 1 or r % 8 or h % 8 or at % 16:
            # a plain clone keeps the strides of dimensions of one, whatever they are
            t = t.clone(memory_format=torch.contiguous_format)
            r, h, d = t.stride()
            at = t.data_ptr()
        return t, _pack_rows(at, r, h), shape


def cache_write(cache, k, v, table, lengths, cu=None):
    """Quantises keys and values [rows, heads, dim] into the cache's pages."""
    if _current_gpu() != cache._index:
        with torch.cuda.device(cache._index):
            return cache_write(cache, k, v, table, lengths, cu)
    k, kr, k_shape = cache._rows(k, cache.heads, "k")
    v, vr, v_shape = cache._rows(v, cache.heads, "v")
    if k_shape != v_shape:
        raise ValueError("one value row for each key row")
    s = cache._seqs(table, lengths, cu, k_shape[0])
    _check(cache._lib.ltc_cache_write(cache._ref, s, kr, vr, _raw_stream(cache._index)), "cache_write")


def cache_read(cache, table, lengths, cu=None, rows=None):
    """The keys and values (two tensors [rows, heads, dim] of the cache's
    dtype) at the positions of the call's rows; rows = cu[-1], which only the
    GPU knows, has to be given with cu."""
    if _current_gpu() != cache._index:
        with torch.cuda.device(cache._index):
            return cache_read(cache, table, lengths, cu, rows)
    if rows is None:
        if cu is not None:
            raise ValueError("rows must be given with cu")
        rows = lengths.numel()
    s = cache._seqs(table, lengths, cu, rows)
    k = torch.empty((rows, cache.heads, cache.dim), dtype=cache.dtype, device=cache.device)
    v = torch.empty_like(k)
    _check(cache._lib.ltc_cache_read(cache._ref, s, k.data_ptr(), v.data_ptr(), _raw_stream(cache._index)),
           "cache_read")
    return k, v


def cache_attend(cache, q, table, lengths, cu=None, window=0, scale=None):
    """softmax(scale * q k^T) v of queries [rows, q_heads, dim] over the
    positions up to each row's own (with window: the last `window` of them);
    zeros for a row that sees nothing.  scale is dim^-0.5 by default.  A call
    is planned for sequences of about its mean: a prompt, or a context of many
    times the others' length, is faster in a call of its own."""
    if _current_gpu() != cache._index:
        with torch.cuda.device(cache._index):
            return cache_attend(cache, q, table, lengths, cu, window, scale)
    if not 0 <= window < 1 << 31:  # ctypes would take it modulo 2^32
        raise LTCError(-1, f"window {window}")
    q, qr, (rows, q_heads, dim) = cache._rows(q, None, "q")
    s = cache._seqs(table, lengths, cu, rows)
    out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=q.device)
    stream = _raw_stream(cache._index)
    need = cache._lib.ltc_cache_attend_workspace_size(cache._ref, s, q_heads, window)
    scale = dim ** -0.5 if scale is None else scale
    if not need:
        _check(cache._lib.ltc_cache_attend(cache._ref, s, qr, q_heads, window, scale, out.data_ptr(), None, 0, stream),
               "cache_attend")
        return out
    # without the lock another thread's call on this stream could replace the
    # workspace, and its memory could be handed out again before this launch
    with cache._lock:
        ws = cache._workspace(need, stream)
        _check(cache._lib.ltc_cache_attend(cache._ref, s, qr, q_heads, window, scale, out.data_ptr(), ws.data_ptr(),
                                           ws.numel(), stream), "cache_attend")
    return out
