"""Attention of many rows at once over the 8-bit cache: calls with enough rows
and workgroups for the kernel that shares positions between four waves, and
scales that lie so far apart that weights leave fp32's range."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, Setup, check_attend, close, ltc  # noqa: F401

pytestmark = pytest.mark.gpu

# heads, group, dim, page, codes, dtype, sequences, rows of each (low, high), positions before them
SHAPES = {
    "64": (16, 16, 64, 16, "e4m3", BF, 24, (4, 12), (0, 150)),
    "64 int8": (13, 16, 64, 64, "int8", FP, 33, (4, 9), (0, 90)),
    "96": (16, 16, 96, 32, "e4m3", FP, 20, (8, 15), (0, 100)),
    "128": (16, 16, 128, 64, "e4m3", BF, 16, (12, 17), (0, 140)),
    "128 odd": (9, 15, 128, 16, "int8", BF, 21, (13, 20), (0, 100)),
    "192": (6, 16, 192, 128, "e4m3", BF, 14, (20, 26), (0, 90)),
    "256": (8, 16, 256, 32, "int8", FP, 9, (28, 35), (0, 70)),
}


def setup(ltc, name, seed, **kw):  # noqa: F811
    H, G, D, P, codes, dtype, n, rows, past = SHAPES[name]
    rng = np.random.default_rng(seed)
    new = [int(rng.integers(rows[0], rows[1] + 1)) for _ in range(n)]
    before = [int(rng.integers(past[0], past[1] + 1)) for _ in range(n)]
    new[1], before[2] = 0, 0
    new[0] += rows[1]
    assert sum(new) * G // n > (64 if D <= 96 else 128) and (sum(new) * G // 128 + n) * H >= (512 if D <= 128 else 256)
    return Setup(ltc, seed, H, D, P, codes, dtype, new, before, **kw), H * G


@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("name", list(SHAPES))
def test_attend(ltc, name, window):  # noqa: F811
    banner(f"attend tiles {name} window {window}")
    s, q_heads = setup(ltc, name, 51)
    check_attend(ltc, s, q_heads, window)


@pytest.mark.parametrize("window", [0, 20])
def test_hidden_nan(ltc, window):  # noqa: F811
    """A NaN among the cached numbers reaches the rows that see it, and a NaN in
    a query its own row."""
    banner(f"nan, window {window}")
    s, q_heads = setup(ltc, "64", 52)
    for i in range(0, len(s.lengths), 2):
        n, new = s.lengths[i], int(s.cu[i + 1] - s.cu[i])
        for t, d, which in ((n - new + 2, 5, "v"), (n - 1, 63, "v"), (n // 3, 1, "v"), (n // 2, 2, "k")):
            if t < n:
                s.o[which][s.table[i, t // 16], i % 16, t % 16, d] = 0x7f if d % 2 else 0xff
    s.upload(ltc)
    q, q64 = s.rows16(q_heads, 1.0)
    q[3, 7, 9], q64[3, 7, 9] = float("nan"), float("nan")
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
    want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu, window)
    assert np.isnan(want).any() and not np.isnan(want).all()
    close(out, want, np.where(np.isnan(slack), 0.0, slack), BF)


def test_bad_pages_and_sequences(ltc):  # noqa: F811
    banner("bad pages")
    s, q_heads = setup(ltc, "64", 53, nan_behind=False)
    s.table[0, 0] = -1
    s.table[4, 1] = len(s.o["scales"])
    s.table[5, 0] = 2 ** 31 - 1
    s.lengths[7] = s.table.shape[1] * 16 + 1
    s.lengths[9] = int(s.cu[10] - s.cu[9]) - 1  # fewer positions than rows
    s.upload(ltc)
    q, q64 = s.rows16(q_heads, 1.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, status = co.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, BF)
    assert int(s.cache.status.item()) == status == 3


def far_scales(s, heads):
    """Value scales of 2^-100 and 2^23 by turns: a page of the small ones has
    weights 2^-123 of the others', and as much of the denominator."""
    s.o["scales"][:, :, 1] = np.where(s.rng.random(s.o["scales"].shape[:2]) < 0.5, 27, 150)


def test_far_scales(ltc):  # noqa: F811
    banner("far scales, tiles")
    s, q_heads = setup(ltc, "64", 54)
    far_scales(s, q_heads)
    s.upload(ltc)
    check_attend(ltc, s, q_heads)


@pytest.mark.parametrize("new,past,single", [([1, 1, 1], [300, 60, 900], True), ([5, 33], [200, 700], False)])
def test_far_scales_few_rows(ltc, new, past, single):  # noqa: F811
    banner(f"far scales, {new} after {past}")
    for seed in range(4):
        s = Setup(ltc, 60 + seed, 2, 64, 16, "e4m3", BF, new, past, single=single)
        far_scales(s, 8)
        s.upload(ltc)
        check_attend(ltc, s, 8)


def test_queries_far_below_one(ltc):  # noqa: F811
    """Queries near bfloat16's smallest normal numbers against keys of large
    scales: the scores are ordinary numbers."""
    s = Setup(ltc, 70, 2, 64, 16, "e4m3", BF, [1, 40], [200, 30])
    s.o["scales"][:, :, 0] = 240  # 2^113
    s.upload(ltc)
    q, q64 = s.rows16(4, 2.0 ** -119)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, BF)
    assert len(np.unique(want.round(3))) > 100


def test_more_positions_than_a_sequence_may_have(ltc):  # noqa: F811
    """A table for more than 2^30 positions, all on one page: lengths past that
    are refused on the device, shorter ones are served."""
    s = Setup(ltc, 71, 1, 64, 256, "e4m3", BF, [1, 1, 1], [299, 40, 9], nan_behind=False, single=True)
    wide = torch.zeros((3, (1 << 22) + 5), dtype=torch.int32, device="cuda")
    wide[:, :s.gtable.shape[1]] = s.gtable
    lengths = torch.tensor([300, (1 << 30) + 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    q, _ = s.rows16(2)
    out = ltc.cache_attend(s.cache, q, wide, lengths)
    want = ltc.cache_attend(s.cache, q[:1], s.gtable[:1], lengths[:1])
    assert not out[1:].any() and int(s.cache.status.item()) == 2
    assert (out[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want.abs().max()
    k, v = ltc.cache_read(s.cache, wide, lengths)
    assert not k[1:].any() and not v[1:].any() and k[0].any()


def test_no_pages(ltc):  # noqa: F811
    cache = ltc.KVCache.empty(0, 2, 64, page=16)
    x = torch.ones((3, 2, 64), dtype=BF, device="cuda")
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    lengths, cu = torch.tensor([9], dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    ltc.cache_write(cache, x, x, table, lengths, cu)
    assert not ltc.cache_attend(cache, x, table, lengths, cu).any()
    assert not ltc.cache_read(cache, table, lengths, cu, rows=3)[0].any()
    with pytest.raises(ltc.LTCError):
        cache.check()
