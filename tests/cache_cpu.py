"""The key/value cache's binding without a GPU: a KVCache over CPU tensors
whose library calls go to functions of the test."""
import types

import torch

from lossless_tensor_compression_amd import kv_cache as kc

GPU = -1  # what Tensor.get_device() says of a CPU tensor


def cpu_cache(monkeypatch, pages=3, heads=2, dim=64, page=16, dtype=torch.bfloat16, **calls):
    """calls: the library's functions by name; those that are not given return 0."""
    monkeypatch.setattr(kc, "_current_gpu", lambda: GPU)
    monkeypatch.setattr(kc, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    names = ("ltc_cache_write", "ltc_cache_read", "ltc_cache_attend", "ltc_cache_attend_workspace_size")
    library = types.SimpleNamespace(**{n: calls.get(n, lambda *a: 0) for n in names})
    monkeypatch.setattr(kc, "lib", lambda: library)

    class OnCpu(torch.Tensor):
        """Says that it is on a GPU, where the constructor asks."""
        is_cuda = True

    def tensor(*shape):
        return torch.zeros(shape, dtype=torch.uint8).as_subclass(OnCpu)

    cache = kc.KVCache(tensor(pages, heads, page // 16, dim // 16, 16, 16), tensor(pages, heads, page // 16, dim, 16),
                       tensor(pages, heads, 2), dtype, "e4m3")
    cache._index = GPU
    return cache


def sequences(lengths, width=4):
    """table and lengths of a call without cu."""
    return (torch.zeros((len(lengths), width), dtype=torch.int32), torch.tensor(lengths, dtype=torch.int32))
