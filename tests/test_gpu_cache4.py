"""The cache of 4-bit codes on the GPU against the 64-bit oracle
(cache4_oracle.py): codes, exponents and drops bit for bit, rows read back to
half a step of their type, attention within the oracle's slack and half a
step."""
import numpy as np
import pytest
import torch

import cache4_oracle as c4
from cache4_setup import Setup4, check_attend4, close
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


# heads, dim, page, dtype, new rows, positions before them
SPANS = {
    "one token, empty page": (2, 64, 16, BF, [1, 1, 1], [0, 16, 32]),
    "one token, begun page": (3, 96, 32, FP, [1, 1, 1, 1], [1, 31, 33, 95]),
    "ragged": (2, 128, 64, BF, [1, 17, 64, 65, 130, 3], [0, 5, 0, 63, 64, 200]),
    "ragged fp16": (5, 64, 16, FP, [15, 16, 1, 33, 47], [1, 0, 15, 16, 2]),
    "no rows": (1, 192, 128, FP, [0, 5, 0, 0, 129, 0], [7, 3, 0, 128, 127, 1]),
    "large heads": (1, 256, 256, FP, [300, 2], [5, 254]),
    "wide page": (2, 256, 128, BF, [131, 1], [0, 127]),
    "many": (1, 64, 16, FP, [(i * 7) % 5 for i in range(150)], [(i * 3) % 40 for i in range(150)]),
    "odd heads": (7, 96, 64, BF, [70, 1, 9], [3, 77, 0]),
    "192": (2, 192, 32, BF, [40, 1], [3, 77]),
}


@pytest.mark.parametrize("case", list(SPANS))
def test_write(ltc, case):
    H, D, P, dtype, new, past = SPANS[case]
    banner(f"write {case}")
    s = Setup4(ltc, 11, H, D, P, dtype, new, past)
    for size in (1.0, 40.0):  # the second write lies in the same places with larger numbers: nothing else changes
        # channels of very different sizes, so that the blocks of a key leave bits unused
        factor = torch.exp2(torch.from_numpy(s.rng.integers(-12, 5, (1, H, D // 32, 1)).repeat(32, -1).reshape(1, H, D))).cuda()
        k = (s.rows16(H, size)[0] * factor).to(dtype)
        v, v64 = s.rows16(H, 0.3 * size)
        ltc.cache_write(s.cache, k, v, s.gtable, s.glengths, s.gcu)
        s.o, status = c4.write(s.o, k.double().cpu().numpy(), v64, s.table, s.lengths, s.cu)
        s.same(s.o)
        assert int(s.cache.status.item()) == status == 0


@pytest.mark.parametrize("dtype", [BF, FP])
def test_write_extremes(ltc, dtype):
    """Zeros, signed zeros, subnormals, the type's largest numbers, infinities
    and NaN; exact borders of a scale; every tie."""
    s = Setup4(ltc, 6, 1, 128, 16, dtype, [16] * 8, [0] * 8)
    x = s.rows16(1)[0].cpu().double()
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -24
    x[0:16] = 0.0
    x[16:32] = -0.0
    x[20, 0, 40] = 1.0
    x[32:48] = tiny * torch.randint(-3, 4, (16, 1, 128))
    x[48:64] *= big / 8
    x[50, 0, 3], x[51, 0, 4] = big, -big
    x[64:80, 0, 5] = float("inf")
    x[65, 0, 6], x[66, 0, 7] = -float("inf"), float("nan")
    x[67, 0, 64:] = float("-inf")
    x[80:96] = float("nan")
    x[90:96] = float("inf")
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0], dtype=torch.float64)
    for i in range(16):  # at many scales, the blocks' own among them
        row = torch.cat([ties, -ties, ties, -ties]).repeat(4)
        row[0::32] = 6.0
        step = torch.tensor([0, 1, 5, 9]).repeat_interleave(32)
        x[96 + i, 0] = row * torch.exp2(-step.double()) * 2.0 ** (i - 8)
    x[112:128] = torch.randint(0, 33, (16, 1, 128)) / 2.0
    x[112, 0, 0], x[113, 0, 0] = 24.0, 24.125  # fits a scale of 4 exactly; just past it
    x = x.to(dtype)
    x64 = x.double().numpy()
    ltc.cache_write(s.cache, x.cuda(), x.cuda(), s.gtable, s.glengths, s.gcu)
    s.o, _ = c4.write(s.o, x64, x64, s.table, s.lengths, s.cu)
    s.same(s.o)


def test_write_strided_rows(ltc):
    """Keys and values as parts of one tensor of queries, keys and values."""
    s = Setup4(ltc, 7, 2, 128, 32, BF, [5, 40], [30, 1])
    qkv = torch.randn(s.rows, 8, 128, device="cuda").to(BF)
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    ltc.cache_write(s.cache, k, v, s.gtable, s.glengths, s.gcu)
    s.o, _ = c4.write(s.o, k.double().cpu().numpy(), v.double().cpu().numpy(), s.table, s.lengths, s.cu)
    s.same(s.o)


@pytest.mark.parametrize("case", list(SPANS))
def test_read(ltc, case):
    H, D, P, dtype, new, past = SPANS[case]
    banner(f"read {case}")
    s = Setup4(ltc, 12, H, D, P, dtype, new, past, spread=6, most_drop=15)
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
    wk, wv, status = c4.read(s.o, s.table, s.lengths, s.cu, s.rows)
    close(k, wk, 0.0, dtype)
    close(v, wv, 0.0, dtype)
    assert int(s.cache.status.item()) == status == 0


def test_single_rows(ltc):
    """Without row offsets: a token of each of 70 sequences, written and read."""
    s = Setup4(ltc, 13, 3, 128, 64, BF, [1] * 70, [(i * 13) % 150 for i in range(70)], single=True)
    k, k64 = s.rows16(3)
    v, v64 = s.rows16(3)
    ltc.cache_write(s.cache, k, v, s.gtable, s.glengths)
    s.o, _ = c4.write(s.o, k64, v64, s.table, s.lengths)
    s.same(s.o)
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths)
    wk, wv, _ = c4.read(s.o, s.table, s.lengths, None, s.rows)
    close(k, wk, 0.0, BF)
    close(v, wv, 0.0, BF)


@pytest.mark.parametrize("group", [1, 3, 16])
@pytest.mark.parametrize("case", list(SPANS))
def test_attend(ltc, case, group):
    H, D, P, dtype, new, past = SPANS[case]
    banner(f"attend {case} group {group}")
    check_attend4(ltc, Setup4(ltc, 14, H, D, P, dtype, new, past), H * group)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1 << 30])
@pytest.mark.parametrize("dtype,dim,page", [(BF, 128, 64), (FP, 64, 16)])
def test_attend_window(ltc, dtype, dim, page, window):
    banner(f"attend window {window}")
    check_attend4(ltc, Setup4(ltc, 15, 2, dim, page, dtype, [1, 70, 5, 130], [300, 100, 0, 64]), 4, window)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("dtype,dim,group", [(BF, 128, 4), (FP, 96, 1), (FP, 256, 7), (BF, 192, 8)])
def test_attend_single_rows(ltc, dtype, dim, group, length):
    banner(f"attend one row at length {length}, dim {dim}")
    s = Setup4(ltc, length, 2, dim, 32, dtype, [1, 1, 1], [length - 1, length // 2, 0], single=True)
    check_attend4(ltc, s, 2 * group)
    check_attend4(ltc, s, 2 * group, window=40)


def test_attend_long(ltc):
    """One row over a long context, split over many workgroups."""
    check_attend4(ltc, Setup4(ltc, 3, 1, 64, 64, BF, [1], [40000], single=True), 2)
    check_attend4(ltc, Setup4(ltc, 3, 1, 128, 128, FP, [3, 1], [20000, 10]), 4)


@pytest.mark.parametrize("new,past", [([200], [0]), ([129, 300], [700, 0]), ([64, 1, 257], [64, 500, 31])])
@pytest.mark.parametrize("dtype,dim,page,heads,group", [(BF, 128, 64, 1, 4), (FP, 64, 16, 2, 1), (FP, 256, 128, 1, 5),
                                                        (BF, 96, 32, 1, 7), (BF, 192, 256, 1, 2)])
def test_attend_prompts(ltc, dtype, dim, page, heads, group, new, past):
    banner(f"attend prompts {new} after {past}, dim {dim} group {group}")
    s = Setup4(ltc, 21, heads, dim, page, dtype, new, past)
    check_attend4(ltc, s, heads * group)
    check_attend4(ltc, s, heads * group, window=90)


@pytest.mark.parametrize("heads,dim,group,new,past", [(8, 64, 8, [130, 9, 260], [100, 0, 3]), (8, 128, 8, [130, 260], [64, 7]),
                                                      (16, 96, 8, [150, 40], [3, 70]), (8, 192, 8, [140], [60]),
                                                      (8, 256, 8, [140], [60])])
def test_attend_tiles(ltc, heads, dim, group, new, past):
    """Enough rows and heads for the kernel whose waves share the positions."""
    banner(f"attend tiles, dim {dim}")
    s = Setup4(ltc, 22, heads, dim, 32, BF if dim != 96 else FP, new + [64] * 12, past + [5] * 12)
    check_attend4(ltc, s, heads * group)


@pytest.mark.parametrize("spread", [8, 40, 100])
@pytest.mark.parametrize("new,past", [([1, 5], [300, 200]), ([140], [300])])
def test_attend_far_scales(ltc, spread, new, past):
    """Scales of neighbouring tokens many powers of two apart, and tokens of
    zeros at the lowest scale."""
    s = Setup4(ltc, 31, 1, 64, 16, BF, new, past)
    ve = s.o["ve"]
    ve[:] = s.rng.integers(127 - spread, 127 + spread // 3, ve.shape)
    zero = s.rng.random(ve.shape) < 0.3
    s.o["k"][zero], s.o["v"][zero] = 0, 0
    s.o["ke"][zero], ve[zero] = 27, 27
    s.upload(ltc)
    check_attend4(ltc, s, 3)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e3])
def test_attend_query_sizes(ltc, size):
    for new, past in (([1, 1], [200, 5]), ([150], [10])):
        s = Setup4(ltc, 32, 2, 64, 32, BF, new, past)
        check_attend4(ltc, s, 4, size=size)
        check_attend4(ltc, s, 4, size=size, scale=1.5)


@pytest.mark.parametrize("new,past,group", [([1, 5], [300, 200], 3), ([140], [300], 3), ([300, 9] + [64] * 12, [5] * 14, 8)])
def test_any_bytes_behind_the_end(ltc, new, past, group):
    """Exponents of tokens that no row sees, every byte there is."""
    s = Setup4(ltc, 44, 8 if len(new) > 2 else 1, 64, 64, BF, new, past)
    for i, n in enumerate(s.lengths):
        for name in ("ke", "ve"):
            for h in range(s.H):
                behind = s.o[name][s.table[i, n // 64], h, n % 64:] if n % 64 else s.o[name][s.free[0], h]
                behind[:] = s.rng.permutation(np.arange(256 - max(16, len(behind)), 256))[:len(behind)] if i % 2 else s.rng.integers(0, 256, len(behind))
    s.upload(ltc)
    check_attend4(ltc, s, s.H * group)


@pytest.mark.parametrize("e", [27, 60, 236, 246, 250])
@pytest.mark.parametrize("new,past,group", [([1, 5], [300, 200], 3), ([300, 9] + [64] * 12, [5] * 14, 8)])
def test_values_of_any_size(ltc, new, past, group, e):
    """Value scales near both ends of their range."""
    s = Setup4(ltc, 45, 8 if len(new) > 2 else 1, 64, 32, BF, new, past)
    s.o["ve"][:] = s.rng.integers(e - 2 if e > 27 else e, e + 2, s.o["ve"].shape)
    s.upload(ltc)
    check_attend4(ltc, s, s.H * group)


def test_key_scales_far_from_one(ltc):
    """Keys of 2^80 under queries of 2^-80, and the other way round: the scores
    are ordinary."""
    for e, size in ((80, 2.0 ** -80), (-80, 2.0 ** 80), (100, 2.0 ** -100), (-96, 2.0 ** 100)):
        for new, past in (([1, 3], [90, 200]), ([140], [30])):
            s = Setup4(ltc, 35, 1, 128, 16, BF, new, past)
            for i, n in enumerate(s.lengths):
                for j in range(-(-n // 16)):
                    s.o["ke"][s.table[i, j]] = (s.o["ke"][s.table[i, j]].astype(int) + e).clip(0, 255)
            s.upload(ltc)
            check_attend4(ltc, s, 4, size=size)


def test_small_drops_reach_the_scores(ltc):
    """Blocks of keys 2^-15 of the largest one, which alone meet the query."""
    for new, past in (([1], [100]), ([140], [30])):
        s = Setup4(ltc, 36, 1, 128, 16, BF, new, past)
        s.o["drops"][..., 0], s.o["drops"][..., 1:] = 0, 15
        s.upload(ltc)
        q, q64 = s.rows16(2, 2.0 ** 14)
        q[..., :32], q64[..., :32] = 0, 0
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        want, slack, _, _, _ = c4.attend4(s.o, q64, s.table, s.lengths, s.cu)
        close(out, want, slack, BF)


# calls of many rows: whose bf16 queries of 128 and 256 dims go in as two numbers of 8 bits
MANY = {64: (8, 8, [300, 9] + [64] * 12), 128: (8, 8, [300, 9] + [64] * 12), 256: (8, 8, [150] + [64] * 10)}


@pytest.mark.parametrize("small", [-3, -9, -13, -16, -20])
@pytest.mark.parametrize("dim", [128, 256])
def test_numbers_far_below_their_head_s_largest(ltc, dim, small):
    """Queries with one large number, which meets keys of zero, and small ones that make the scores."""
    heads, group, new = MANY[dim]
    s = Setup4(ltc, 37, heads, dim, 32, BF, new, [5] * len(new))
    s.o["k"][..., 7] = 0
    s.upload(ltc)
    q, _ = s.rows16(heads * group, 2.0 ** small)
    q[..., 7] = 1.5
    # scores of ordinary size
    scale = dim ** -0.5 * 2.0 ** -small
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, scale=scale)
    want, slack, _, _, status = c4.attend4(s.o, q.double().cpu().numpy(), s.table, s.lengths, s.cu, 0, scale, 2.0 ** -21)
    close(out, want, slack, BF)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_odd_queries_of_many_rows_stay_in_their_rows(ltc, dim, bad):
    heads, group, new = MANY[dim]
    s = Setup4(ltc, 38, heads, dim, 32, BF, new, [5] * len(new))
    q, _ = s.rows16(heads * group, 1.0)
    plain = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    q[3, 5, 9] = q[70, 0, dim - 1] = bad
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    nan = torch.isnan(out)
    for r, h in ((3, 5), (70, 0)):
        assert nan[r, h].all()
        out[r, h] = plain[r, h]
    assert torch.equal(out, plain) and int(nan.sum()) == 2 * dim


@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100])
def test_queries_of_any_size_of_many_rows(ltc, size):
    """Their power of two goes into the products, as far as fp32 has it."""
    heads, group, new = MANY[128]
    s = Setup4(ltc, 39, heads, 128, 32, BF, new, [5] * len(new))
    e = round(np.log2(size))
    for i, n in enumerate(s.lengths):
        for j in range(-(-n // 32)):
            s.o["ke"][s.table[i, j]] = (s.o["ke"][s.table[i, j]].astype(int) - e).clip(30, 250)
    s.upload(ltc)
    q, q64 = s.rows16(heads * group, size)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    # queries of 2^-130 are subnormal: their 8 bits are fewer, and exact all the same
    want, slack, _, _, _ = c4.attend4(s.o, q64, s.table, s.lengths, s.cu, query_error=2.0 ** -21 if size > 2.0 ** -115 else 2.0 ** -8)
    close(out, want, slack, BF)


@pytest.mark.parametrize("new,past,heads,group", [([1, 1, 1], [70, 80, 5], 1, 4), ([5, 9], [30, 40], 2, 4)])
def test_infinite_queries_of_few_rows(ltc, new, past, heads, group):
    """One row's infinity makes it NaN, whatever the signs of what it meets."""
    for sign in (1, -1):
        s = Setup4(ltc, 40, heads, 64, 32, BF, new, past)
        s.o["k"][..., 7] = 3  # all positive: scores of one infinity
        s.upload(ltc)
        q, _ = s.rows16(heads * group, 1.0)
        plain = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        q[1, 1, 7] = sign * float("inf")
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        assert torch.isnan(out[1, 1]).all()
        out[1, 1] = plain[1, 1]
        assert torch.equal(out, plain)


def test_query_nan_stays_in_its_row(ltc):
    for new, past in (([1, 1, 1], [70, 80, 5]), ([150], [10])):
        s = Setup4(ltc, 34, 1, 64, 32, FP, new, past)
        q, q64 = s.rows16(4, 1.0)
        q[0, 1, 7], q64[0, 1, 7] = float("nan"), float("nan")
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        want, slack, _, _, _ = c4.attend4(s.o, q64, s.table, s.lengths, s.cu)
        assert np.isnan(want).sum() == 64
        close(out, want, np.where(np.isnan(slack), 0.0, slack), FP)


def test_bad_pages_and_sequences(ltc):
    """Table entries outside the cache, lengths past the table, fewer positions
    than rows: nothing else changes, the status says so."""
    s = Setup4(ltc, 41, 2, 64, 16, BF, [20, 5, 33, 4, 7], [30, 0, 40, 9, 3])
    s.table[0, 2] = -1
    s.table[2, 4] = s.pages
    s.table[2, 1] = 2 ** 31 - 1
    s.lengths[3] = s.table.shape[1] * 16 + 1
    s.lengths[4] = 6
    s.upload(ltc)
    q, q64 = s.rows16(4, 1.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, _, _, status = c4.attend4(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, BF)
    assert int(s.cache.status.item()) == status == 3
    with pytest.raises(ltc.LTCError):
        s.cache.check()
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
    wk, wv, status = c4.read(s.o, s.table, s.lengths, s.cu, s.rows)
    close(k, wk, 0.0, BF)
    close(v, wv, 0.0, BF)
    assert int(s.cache.status.item()) == status == 3
    s.cache.status.zero_()
    k, k64 = s.rows16(2)
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    s.o, status = c4.write(s.o, k64, k64, s.table, s.lengths, s.cu)
    s.same(s.o)
    assert int(s.cache.status.item()) == status == 3


def test_empty_cache_is_zeros(ltc):
    cache = ltc.KVCache.empty(5, 2, 96, page=16, codes="e2m1")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lengths, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([50], [0, 50]))
    for x in ltc.cache_read(cache, table, lengths, cu, rows=50):
        assert not x.any()
    assert not ltc.cache_attend(cache, torch.randn(50, 2, 96, device="cuda").to(BF), table, lengths, cu).any()
    cache.check()


def test_rows_of_no_sequence(ltc):
    """Rows in front of cu[0] and behind cu[-1] come out as zeros."""
    s = Setup4(ltc, 43, 2, 128, 32, BF, [5, 3], [20, 70])
    cu = torch.tensor([2, 7, 10], dtype=torch.int32, device="cuda")
    q = torch.randn(14, 4, 128, device="cuda").to(BF)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, cu)
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths, cu, rows=14)
    inner = ltc.cache_attend(s.cache, q[2:10], s.gtable, s.glengths, s.gcu)
    for x in (out, k, v):
        assert not x[:2].any() and not x[10:].any() and x[2:10].any()
    assert torch.equal(out[2:10], inner)
