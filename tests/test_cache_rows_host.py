"""What the key/value cache's binding hands to the library for rows of all
strides, without a GPU: strides that the library takes, and the same numbers."""
import ctypes
import struct

import pytest
import torch

from cache_cpu import cpu_cache, sequences
from lossless_tensor_compression_amd import kv_cache as kc


def numbers(packed, shape):
    """The 16-bit numbers of an ltc_cache_rows, checked as the library does."""
    base, r, h = struct.unpack("=QQQ", packed)
    assert base % 16 == 0 and r % 8 == 0 and h % 8 == 0
    return [[list((ctypes.c_uint16 * shape[2]).from_address(base + 2 * (i * r + j * h))) for j in range(shape[1])]
            for i in range(shape[0])]


def views():
    x = torch.randn(5, 3 * 1027).to(torch.bfloat16)
    yield "one row of a product of odd width", x[:, :128].unflatten(1, (2, 64))[1:2]
    yield "rows of a product of odd width", x[:, :128].unflatten(1, (2, 64))[1:4]
    yield "one row, misaligned", x[:, 5:133].unflatten(1, (2, 64))[2:3]
    yield "one head of odd stride", torch.as_strided(x, (3, 1, 64), (64, 13, 1), 8)
    yield "one row and head of odd strides", torch.as_strided(x, (1, 1, 64), (77, 13, 1), 8)
    yield "transposed", torch.randn(64, 2, 3).to(torch.bfloat16).permute(2, 1, 0)
    yield "one row for all", torch.randn(1, 2, 64).to(torch.bfloat16).expand(4, 2, 64)
    yield "contiguous", torch.randn(3, 2, 64).to(torch.bfloat16)


@pytest.mark.parametrize("name,x", list(views()))
def test_rows(monkeypatch, name, x):
    got = []
    cache = cpu_cache(monkeypatch, heads=x.shape[1],
                      ltc_cache_write=lambda ref, s, k, v, stream: got.extend([numbers(k, x.shape), numbers(v, x.shape)]) or 0,
                      ltc_cache_attend=lambda ref, s, q, *a: got.append(numbers(q, x.shape)) or 0)
    want = (x.contiguous().view(torch.int16).int() & 0xffff).tolist()
    table, lengths = sequences([9] * len(x))
    kc.cache_write(cache, x, x, table, lengths)
    kc.cache_attend(cache, x, table, lengths)
    assert len(got) == 3 and all(g == want for g in got)
