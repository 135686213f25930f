"""A paged key/value cache in 8 or 4 bits: quantised as it is written, read
back, attended to in place, and cut to the positions that were worth most.

  KVCache.empty(...) / KVCache.of(...)  the cache's tensors and their layout
  cache_write(cache, k, v, table, lengths, cu)   new keys and values to their positions
  cache_read(cache, table, lengths, cu, rows)    positions back as 16-bit rows
  cache_attend(cache, q, table, lengths, cu)     attention of new queries; with
                                                 weights=, what each position got is added up
  cache_evict(cache, weights, table, lengths, to, keep, recent)
                                                 the positions of most weight to other pages

A binding over ltc_cache_write, ltc_cache_read, ltc_cache_attend,
ltc_cache_attend_weigh and ltc_cache_evict of include/ltc.h, where the layouts,
the rounding and what happens with bad tables are written down.  Calls run on
the current stream, allocate nothing but their outputs and a workspace, which a
GPU's caches keep together for each stream (attention with weights of few rows
wants up to 128 MiB, others a few), and never synchronise, so they can be
captured in a graph.  They have no backward pass: rows that require a gradient
are refused.  Threads may share a cache; their calls on one stream run in the
order in which they are made.

Rows cu[i]..cu[i+1] of a call belong to sequence i and stand for its last
positions, lengths[i] - (cu[i+1] - cu[i]) to lengths[i] - 1; without cu each
sequence has one row.  Rows outside cu[0]..cu[-1] belong to no sequence and
come out as zeros.  Position t of sequence i is token t % page of page
table[i, t // page].  table, lengths and cu are int32 tensors on the GPU.
"""
import ctypes
import struct
import threading
import weakref

import torch

from . import LTCError, _check, lib

E4M3, INT8, E2M1 = 0, 1, 3
CODES = {"e4m3": E4M3, "int8": INT8, "e2m1": E2M1}
CACHE_DTYPES = {torch.bfloat16: 1, torch.float16: 2}
PAGES = (16, 32, 64, 128, 256)
DIMS = (64, 96, 128, 192, 256)
DROP_BYTES = {64: 1, 96: 2, 128: 2, 192: 4, 256: 4}  # a token's, of E2M1 codes
BAD_PAGE, BAD_SEQUENCE = 1, 2
WS_ZEROS = 65536

_INT32 = torch.int32
_current_gpu = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() builds a Stream object: 2.7 us a call
_pack_seqs = struct.Struct("=QQQQIIII").pack      # ltc_cache_seqs
_pack_rows = struct.Struct("=QQQ").pack           # ltc_cache_rows


_lock = threading.Lock()  # from a workspace's lookup to the launch that uses it
_workspaces = weakref.WeakValueDictionary()  # (GPU, stream) -> the workspace that its caches share


def _room(need):
    """Bytes of a workspace of at least `need`: a power of two, and from 16 MiB on the next eighth of one."""
    bits = (need - 1).bit_length()
    step = 1 << (bits if bits <= 24 else bits - 4)
    return -(-need // step) * step


class CacheStruct(ctypes.Structure):
    _fields_ = [("d_k_codes", ctypes.c_void_p), ("d_v_codes", ctypes.c_void_p), ("d_scales", ctypes.c_void_p),
                ("d_status", ctypes.c_void_p), ("pages", ctypes.c_uint32), ("heads", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("page", ctypes.c_uint32), ("codes", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def _take_rows(t, heads, dim, name):
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which the cache's operators have not: call under torch.no_grad()")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [rows, {'heads' if heads is None else heads}, {dim}]")
    r, h, d = t.stride()
    at = t.data_ptr()
    if d != 1 or r % 8 or h % 8 or at % 16:
        # a plain clone keeps the strides of dimensions of one, whatever they are
        t = t.clone(memory_format=torch.contiguous_format)
        r, h, d = t.stride()
        at = t.data_ptr()
    return t, _pack_rows(at, r, h), shape


class KVCache:
    """The tensors of a cache and what the library has to know of them.

    k_codes uint8 [pages, heads, page/16, dim/16, 16 tokens, 16 dims]
    v_codes uint8 [pages, heads, page/16, dim, 16 tokens]
    scales  uint8 [pages, heads, 2], a scale is 2^(byte - 127)
    dtype: torch.bfloat16 or torch.float16, of keys, values, queries and
    outputs; codes: "e4m3", "int8" or, in 4 bits, "e2m1":
    k_codes uint8 [pages, heads, page/16, dim/32, 16 tokens, 16], two dims a byte
    v_codes uint8 [pages, heads, page/16, dim, 8], two tokens a byte
    scales  uint8 [pages, heads, page * (2 + DROP_BYTES[dim])]: exponents of
            the tokens' keys, of their values, and for each token a nibble for
            each 32 dims of its key, how far below its scale theirs is"""

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
        pages, heads, page, dim = self._shape(k_codes, v_codes, scales, codes)
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
        self._lock = _lock

    @staticmethod
    def _shape(k_codes, v_codes, scales, codes):
        four = codes == "e2m1"
        part, tokens = (32, 8) if four else (16, 16)  # dims of 16 bytes of keys, bytes of 16 tokens of values
        if k_codes.dim() != 6 or k_codes.shape[4:] != (16, 16):
            raise ValueError(f"k_codes must be [pages, heads, page/16, dim/{part}, 16, 16]")
        pages, heads, blocks, parts = k_codes.shape[:4]
        if v_codes.shape != (pages, heads, blocks, parts * part, tokens):
            raise ValueError(f"v_codes must be [pages, heads, page/16, dim, {tokens}]")
        if blocks * 16 not in PAGES:
            raise ValueError(f"a page must have one of {PAGES} tokens")
        if parts * part not in DIMS:
            raise ValueError(f"a head must have one of {DIMS} dims")
        wide = blocks * 16 * (2 + DROP_BYTES[parts * part]) if four else 2
        if scales.shape != (pages, heads, wide):
            raise ValueError(f"scales must be [pages, heads, {wide}]")
        if heads < 1:
            raise ValueError("at least one head")
        return pages, heads, blocks * 16, parts * part

    @classmethod
    def of(cls, k_codes, v_codes, scales, dtype=torch.bfloat16, codes="e4m3"):
        """A cache over tensors that the caller holds."""
        return cls(k_codes, v_codes, scales, dtype, codes)

    @classmethod
    def empty(cls, pages, heads, dim, page=64, dtype=torch.bfloat16, codes="e4m3", device="cuda"):
        """A cache with tensors of its own, zeros with the lowest scale."""
        if page not in PAGES or dim not in DIMS:
            raise ValueError(f"page must be one of {PAGES} and dim one of {DIMS}")
        def zeros(*shape):
            return torch.zeros((pages, heads, *shape), dtype=torch.uint8, device=device)

        if codes == "e2m1":
            scales = zeros(page * (2 + DROP_BYTES[dim]))
            scales[..., :2 * page] = 27
            return cls(zeros(page // 16, dim // 32, 16, 16), zeros(page // 16, dim, 8), scales, dtype, codes)
        return cls(zeros(page // 16, dim // 16, 16, 16), zeros(page // 16, dim, 16),
                   torch.full((pages, heads, 2), 27, dtype=torch.uint8, device=device), dtype, codes)

    def no_weights(self):
        """Zeros to add positions' weights to: float32 [pages, heads, page]."""
        return torch.zeros((self.pages, self.heads, self.page), dtype=torch.float32, device=self.device)

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
        it has launched.  A stream's calls run in order, so each stream keeps
        one, for all caches of the GPU; a captured call gets its own, which
        lives and is cleared with the graph."""
        captured = torch._C._cuda_isCurrentStreamCapturing()
        ws = None if captured else self._workspaces.get(stream)
        if ws is not None and ws.numel() >= need:
            return ws
        ws = None if captured else _workspaces.get((self._index, stream))
        if ws is None or ws.numel() < need:
            ws = torch.empty(_room(need), dtype=torch.uint8, device=self.device)
            ws[:WS_ZEROS].zero_()
        if not captured:
            self._workspaces[stream] = _workspaces[self._index, stream] = ws
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

    def _weights(self, t):
        if t.dtype is not torch.float32 or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError("weights must be contiguous float32 on the cache's GPU")
        if t.shape != (self.pages, self.heads, self.page):
            raise ValueError(f"weights must be [{self.pages}, {self.heads}, {self.page}]")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError("weights require a gradient, which the cache's operators have not: call under torch.no_grad()")
        return t.data_ptr()

    def _rows(self, t, heads, name):
        """t as rows that the kernels can take (a copy where its strides or
        alignment do not let them), its ltc_cache_rows as bytes and its shape."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name} must be {self.dtype} on the cache's GPU")
        return _take_rows(t, heads, self.dim, name)


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


def cache_attend(cache, q, table, lengths, cu=None, window=0, scale=None, weights=None):
    """softmax(scale * q k^T) v of queries [rows, q_heads, dim] over the
    positions up to each row's own (with window: the last `window` of them);
    zeros for a row that sees nothing.  scale is dim^-0.5 by default.  A call
    is planned for sequences of about its mean: a prompt, or a context of many
    times the others' length, is faster in a call of its own.

    weights (float32 [pages, heads, page], as KVCache.no_weights() makes them)
    get what each position is worth to the call's rows added to them: at its
    token's place and each of the cache's heads, the softmax's weights of all
    rows that see it and all query heads that read the head.  Those of the
    positions that the rows stand for begin at zero; those that no row sees are
    not touched.  No two sequences of such a call may have rows that see
    positions of the same page.  Where rows are attended to without weights,
    their positions keep what the page's earlier tokens had: clear those of a
    page that is handed out anew then."""
    if _current_gpu() != cache._index:
        with torch.cuda.device(cache._index):
            return cache_attend(cache, q, table, lengths, cu, window, scale, weights)
    if not 0 <= window < 1 << 31:  # ctypes would take it modulo 2^32
        raise LTCError(-1, f"window {window}")
    q, qr, (rows, q_heads, dim) = cache._rows(q, None, "q")
    s = cache._seqs(table, lengths, cu, rows)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)  # half the time of torch.empty with a shape
    stream = _raw_stream(cache._index)
    scale = dim ** -0.5 if scale is None else scale
    if weights is not None:
        at = cache._weights(weights)
        need = cache._lib.ltc_cache_attend_weigh_workspace_size(cache._ref, s, q_heads, window)
        with cache._lock:
            ws = cache._workspace(need, stream) if need else None
            _check(cache._lib.ltc_cache_attend_weigh(cache._ref, s, qr, q_heads, window, scale, out.data_ptr(), at,
                                                     ws.data_ptr() if need else None, ws.numel() if need else 0, stream),
                   "cache_attend")
        return out
    need = cache._lib.ltc_cache_attend_workspace_size(cache._ref, s, q_heads, window)
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


def cache_evict(cache, weights, table, lengths, to, keep, recent=0):
    """Cuts sequences to `keep` positions: the last `recent` ones, and of the
    others those of most weight (of equal ones the first; a NaN is below all
    numbers), each of the cache's heads by itself.  They are moved, in their
    order and with their weights, to the pages that to [sequences, at least
    keep / page] names, whose positions they are from then on: 0 to keep - 1.
    Pages of `to` must not be in use, here or twice; those of table are free
    afterwards.  Windows of later calls count the kept positions.  A sequence of
    no more than `keep` positions keeps all of them.
    4-bit codes are moved as they are; a page of 8-bit ones gets the largest
    scale that its tokens had, and codes of smaller scales are rounded again.

    Returns the new lengths, int32 [sequences], and the kept positions, int32
    [sequences, heads, keep], in order and -1 behind the last."""
    if _current_gpu() != cache._index:
        with torch.cuda.device(cache._index):
            return cache_evict(cache, weights, table, lengths, to, keep, recent)
    if not 1 <= keep < 1 << 31 or not 0 <= recent <= keep:  # ctypes would take them modulo 2^32
        raise LTCError(-1, f"keep {keep}, recent {recent}")
    at, seqs = cache._weights(weights), lengths.numel()
    s = cache._seqs(table, lengths, None, seqs)
    if to.dtype is not _INT32 or to.get_device() != cache._index:
        raise ValueError("to must be int32 on the cache's GPU")
    pages = -(-keep // cache.page)
    if to.dim() != 2 or to.shape[0] != seqs or to.shape[1] < pages:
        raise ValueError(f"to must be [sequences, at least {pages} pages]")
    width = to.shape[1]
    if to.stride(1) != 1 and width > 1:
        raise ValueError("the rows of to must be contiguous")
    step = to.stride(0) if seqs > 1 else width
    if step < width:
        raise ValueError("the rows of to must not overlap")
    new = torch.empty(seqs, dtype=_INT32, device=cache.device)
    positions = torch.empty((seqs, cache.heads, keep), dtype=_INT32, device=cache.device)
    stream = _raw_stream(cache._index)
    need = cache._lib.ltc_cache_evict_workspace_size(cache._ref, s)
    with cache._lock:
        ws = cache._workspace(need, stream) if need else None
        _check(cache._lib.ltc_cache_evict(cache._ref, s, at, to.data_ptr(), step, width, keep, recent, new.data_ptr(),
                                          positions.data_ptr(), ws.data_ptr() if need else None, ws.numel() if need else 0,
                                          stream), "cache_evict")
    return new, positions
