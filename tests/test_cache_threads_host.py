"""Threads that share a key/value cache and a stream, without a GPU: what a
call hands to the library lives until the library has launched."""
import threading
import weakref

import torch

from cache_cpu import cpu_cache, sequences
from lossless_tensor_compression_amd import kv_cache as kc


def test_workspace_outlives_its_launch(monkeypatch):
    """While a call is in the library, another thread's call on the same
    stream needs a larger workspace."""
    made = {}  # pointer -> the workspace's tensor, weakly
    empty = torch.empty

    def recorded(*args, **kw):
        t = empty(*args, **kw)
        if kw["dtype"] == torch.uint8:
            made[t.data_ptr()] = weakref.ref(t)
        return t

    sizes, seen = [100000, 300000], []

    def attend(cache_ref, s, q, q_heads, window, scale, out, ws, size, stream):
        if threading.current_thread() is not other:
            other.start()
            other.join(timeout=0.5)  # it waits for this call, or takes the workspace from under it
        seen.append((size, made[ws]() is not None))
        return 0

    cache = cpu_cache(monkeypatch, ltc_cache_attend=attend,
                      ltc_cache_attend_workspace_size=lambda *a: sizes.pop(0))
    monkeypatch.setattr(torch, "empty", recorded)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    other = threading.Thread(target=lambda: kc.cache_attend(cache, q, *sequences([5])))
    kc.cache_attend(cache, q, *sequences([5]))
    other.join(timeout=10)
    assert not other.is_alive()
    assert all(alive for _, alive in seen), seen
    assert [size for size, _ in seen] == [1 << 17, 1 << 19]
