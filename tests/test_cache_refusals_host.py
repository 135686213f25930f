"""Arguments that the key/value cache's binding refuses by itself, without a
GPU."""
import pytest
import torch

from cache_cpu import cpu_cache, sequences
from lossless_tensor_compression_amd import LTCError
from lossless_tensor_compression_amd import kv_cache as kc


@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 32 + 5, 1 << 31, 2 ** 32, 2 ** 32 + 5, 2 ** 64 + 1])
def test_windows_out_of_range(monkeypatch, window):
    """Not taken modulo 2^32: a window of 2^32 + 5 is not one of 5."""
    reached = []
    cache = cpu_cache(monkeypatch, ltc_cache_attend=lambda *a: reached.append(a) or 0)
    with pytest.raises(LTCError) as e:
        kc.cache_attend(cache, torch.zeros((1, 4, 64), dtype=torch.bfloat16), *sequences([9]), window=window)
    assert e.value.code == -1 and not reached


@pytest.mark.parametrize("window", [0, 1, 2 ** 31 - 1])
def test_windows_in_range(monkeypatch, window):
    reached = []
    cache = cpu_cache(monkeypatch, ltc_cache_attend=lambda *a: reached.append(a[4]) or 0)
    kc.cache_attend(cache, torch.zeros((1, 4, 64), dtype=torch.bfloat16), *sequences([9]), window=window)
    assert reached == [window]


def test_rows_that_require_a_gradient(monkeypatch):
    """An output without one would be detached silently."""
    reached = []
    cache = cpu_cache(monkeypatch, **{n: lambda *a: reached.append(a) or 0 for n in ("ltc_cache_attend", "ltc_cache_write")})
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    w = torch.ones((), dtype=torch.bfloat16, requires_grad=True)
    for leaf in (x.clone().requires_grad_(), x * w):
        with pytest.raises(ValueError, match="gradient"):
            kc.cache_attend(cache, leaf, *sequences([9]))
        for k, v in ((leaf, x), (x, leaf)):
            with pytest.raises(ValueError, match="gradient"):
                kc.cache_write(cache, k, v, *sequences([9]))
        assert not reached
        with torch.no_grad():
            kc.cache_attend(cache, leaf, *sequences([9]))
            kc.cache_write(cache, leaf, leaf, *sequences([9]))
        assert len(reached) == 2
        reached.clear()
        kc.cache_attend(cache, leaf.detach(), *sequences([9]))
        reached.clear()
