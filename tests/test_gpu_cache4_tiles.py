"""Prompts over 4-bit codes through the kernel whose waves share the positions:
every size of a head in fp16, windows, missing pages and value scales far
apart.  Four of a key head's sixteen query heads are compared."""
import numpy as np
import pytest
import torch

import cache4_oracle as c4
from cache4_setup import Setup4, close
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
H, G = 8, 16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def tiles(ltc, dim, dtype, seed, page=16, **kw):
    """Sequences of about 9 rows, 144 packed ones: more than a tile, and tiles for all CUs, whatever a later rule asks
    for (twice as many and more of it)."""
    new = [7 + i % 5 for i in range(64 if dim <= 128 else 32)]
    s = Setup4(ltc, seed, H, dim, page, dtype, new, [(i * 29) % 130 for i in range(len(new))], **kw)
    mean, units = -(-s.rows * G // len(new)), (s.rows * G // 128 + len(new)) * H
    assert mean > 128 and units >= (512 if dim <= 128 else 256)
    return s


def check(ltc, s, window=0, scale=None):
    q, q64 = s.rows16(H * G, 1.5)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, scale=scale)
    some = np.sort(np.concatenate([s.rng.choice(G, 4, False) + h * G for h in range(H)]))
    want, slack, _, _, status = c4.attend4(s.o, q64[:, some], s.table, s.lengths, s.cu, window, scale)
    close(out[:, torch.from_numpy(some).cuda()], want, slack, s.dtype)
    assert int(s.cache.status.item()) == status
    assert not torch.isnan(out).any()
    return status


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_sizes_of_heads(ltc, dim, dtype):
    banner(f"tiles of 4-bit codes, {dtype}, dim {dim}")
    assert check(ltc, tiles(ltc, dim, dtype, 131)) == 0


@pytest.mark.parametrize("dim,dtype,window", [(64, BF, 1), (64, FP, 33), (96, FP, 64), (128, BF, 17), (128, BF, 64), (128, FP, 100),
                                              (192, BF, 40), (256, BF, 70), (256, FP, 16), (128, BF, 2 ** 31 - 1)])
def test_windows(ltc, dim, dtype, window):
    banner(f"tiles of 4-bit codes, {dtype}, dim {dim}, window {window}")
    assert check(ltc, tiles(ltc, dim, dtype, 132), window) == 0


@pytest.mark.parametrize("dim,dtype,page", [(64, FP, 16), (96, BF, 32), (128, BF, 16), (128, FP, 64), (192, FP, 16), (256, BF, 32), (256, FP, 16)])
def test_missing_pages(ltc, dim, dtype, page):
    """Of every third sequence one page, its last or first or one between, and all of some."""
    banner(f"tiles of 4-bit codes, {dtype}, dim {dim}, missing pages")
    s = tiles(ltc, dim, dtype, 133, page)
    for i in range(0, len(s.lengths), 3):
        last = (s.lengths[i] - 1) // page
        s.table[i, (0, last, last // 2)[i // 3 % 3]] = (-1, s.pages, 2 ** 31 - 1)[i // 3 % 3]
    s.table[4, :(s.lengths[4] - 1) // page + 1] = -7
    s.gtable = torch.from_numpy(s.table).cuda()
    assert check(ltc, s) == 1


@pytest.mark.parametrize("spread", [25, 45, 100])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (96, FP), (128, BF), (128, FP), (256, BF)])
def test_value_scales_far_apart(ltc, dim, dtype, spread):
    """Tokens' value scales many powers of two apart, and tokens of zeros at the lowest one."""
    banner(f"tiles of 4-bit codes, {dtype}, dim {dim}, value scales 2^{spread} apart")
    s = tiles(ltc, dim, dtype, 134)
    ve = s.o["ve"]
    # fp16 rows hold values up to 2^15
    ve[:] = s.rng.integers(127 - spread, 127 + min(spread // 3, 10), ve.shape)
    zero = s.rng.random(ve.shape) < 0.3
    s.o["k"][zero], s.o["v"][zero] = 0, 0
    s.o["ke"][zero], ve[zero] = 27, 27
    s.upload(ltc)
    assert check(ltc, s) == 0
