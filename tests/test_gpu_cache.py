"""The 8-bit key/value cache on the GPU against the 64-bit oracle
(cache_oracle.py): codes and scales bit for bit, rows read back to half a
step of their type, attention within the oracle's slack and half a step."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


class Setup:
    """A cache of random codes on both sides, sequences with shuffled pages."""

    def __init__(self, ltc, seed, heads, dim, page, codes, dtype, new, past, spread=1, nan_behind=True, single=False):
        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.codes, self.H, self.D, self.P = dtype, codes, heads, dim, page
        self.lengths = [a + b for a, b in zip(new, past)]
        self.cu = None if single else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = sum(new)
        need = [-(-n // page) for n in self.lengths]
        pages = sum(need) + 2
        width = max(need + [1]) + 1
        order = rng.permutation(pages)
        self.table = rng.integers(-5, pages + 5, (len(new), width)).astype(np.int32)  # behind the end: anything
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        top = 110.0 if codes == "e4m3" else 30.0
        k, v = (co.code(np.clip(rng.normal(0, top, (pages, heads, page, dim)), -co.TOP[codes], co.TOP[codes]), codes)
                for _ in range(2))
        if nan_behind and codes == "e4m3":  # whatever is behind a sequence's end does not count
            for i, n in enumerate(self.lengths):
                if n % page:
                    for x in (k, v):
                        x[self.table[i, n // page], :, n % page:] = 0x7f
            for p in order[at:]:
                k[p], v[p] = 0x7f, 0xff
        middle = 120 if codes == "e4m3" else 122
        scales = rng.integers(middle - spread, middle + spread + 1, (pages, heads, 2)).astype(np.uint8)
        self.o = {"k": k, "v": v, "scales": scales, "codes": codes}
        self.upload(ltc)

    def upload(self, ltc):
        ks, vs = co.to_stored(self.o["k"], self.o["v"])
        self.cache = ltc.KVCache.of(torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda(),
                                    torch.from_numpy(self.o["scales"].copy()).cuda(), dtype=self.dtype, codes=self.codes)
        self.gtable = torch.from_numpy(self.table).cuda()
        self.glengths = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.gcu = None if self.cu is None else torch.from_numpy(self.cu).cuda()

    def rows16(self, heads, size=1.0):
        x = torch.from_numpy(self.rng.normal(0, size, (self.rows, heads, self.D))).to(self.dtype)
        return x.cuda(), x.double().numpy()

    def got(self):
        k, v = co.from_stored(self.cache.k_codes.cpu().numpy(), self.cache.v_codes.cpu().numpy())
        return k, v, self.cache.scales.cpu().numpy()


def close(got, want, slack, dtype):
    """got within slack and half a step of want."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = np.abs(got - want) > slack + HALF[dtype] * (np.abs(want) + slack) + SMALLEST[dtype]
    bad &= ~np.isnan(want)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], np.broadcast_to(slack, got.shape)[bad][:5])


def same_cache(s, want):
    k, v, scales = s.got()
    assert np.array_equal(scales, want["scales"]), np.argwhere(scales != want["scales"])[:5]
    for a, b in ((k, want["k"]), (v, want["v"])):
        if s.codes == "e4m3":  # one NaN is as good as another
            nan = (b & 127) == 127
            assert np.array_equal((a & 127) == 127, nan)
            a, b = np.where(nan, 0, a), np.where(nan, 0, b)
        assert np.array_equal(a, b), np.argwhere(a != b)[:5]


def check_attend(ltc, s, q_heads, window=0, scale=None, size=2.0):
    q, q64 = s.rows16(q_heads, size)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, scale=scale)
    want, slack, status = co.attend(s.o, q64, s.table, s.lengths, s.cu, window, scale)
    close(out, want, slack, s.dtype)
    assert int(s.cache.status.item()) == status == 0


BF, FP = torch.bfloat16, torch.float16
# heads, dim, page, codes, dtype, new rows, positions before them
SPANS = {
    "one token, empty page": (2, 64, 16, "e4m3", BF, [1, 1, 1], [0, 16, 32]),
    "one token, begun page": (3, 96, 32, "int8", FP, [1, 1, 1, 1], [1, 31, 33, 95]),
    "ragged": (2, 128, 64, "e4m3", BF, [1, 17, 64, 65, 130, 3], [0, 5, 0, 63, 64, 200]),
    "ragged int8": (5, 64, 16, "int8", BF, [15, 16, 1, 33, 47], [1, 0, 15, 16, 2]),
    "no rows": (1, 192, 128, "e4m3", FP, [0, 5, 0, 0, 129, 0], [7, 3, 0, 128, 127, 1]),
    "large heads": (1, 256, 256, "int8", FP, [300, 2], [5, 254]),
    "wide page": (2, 256, 128, "e4m3", BF, [131, 1], [0, 127]),
    "many": (1, 64, 16, "e4m3", FP, [(i * 7) % 5 for i in range(150)], [(i * 3) % 40 for i in range(150)]),
    "odd heads": (7, 96, 64, "e4m3", BF, [70, 1, 9], [3, 77, 0]),
}


@pytest.mark.parametrize("case", list(SPANS))
def test_write(ltc, case):
    H, D, P, codes, dtype, new, past = SPANS[case]
    banner(f"write {case}")
    s = Setup(ltc, 11, H, D, P, codes, dtype, new, past, spread=3)
    for size in (1.0, 40.0):  # the second write lies in the same places with larger numbers: scales grow
        k, k64 = s.rows16(H, size)
        v, v64 = s.rows16(H, 0.3 * size)
        ltc.cache_write(s.cache, k, v, s.gtable, s.glengths, s.gcu)
        s.o, status = co.write(s.o, k64, v64, s.table, s.lengths, s.cu)
        same_cache(s, s.o)
        assert int(s.cache.status.item()) == status == 0


@pytest.mark.parametrize("codes,dtype", [("e4m3", BF), ("int8", FP), ("e4m3", FP), ("int8", BF)])
def test_write_single_rows_grow_a_page(ltc, codes, dtype):
    """Tokens one at a time, without row offsets, each larger than the last:
    codes are halved and rounded again and again."""
    s = Setup(ltc, 5, 2, 64, 16, codes, dtype, [1, 1], [0, 7], single=True)
    lengths = np.array(s.lengths)
    for step in range(8):
        k, k64 = s.rows16(2, 1.5 ** step)
        v, v64 = s.rows16(2, 1.3 ** step)
        s.lengths = list(lengths + step)
        s.glengths = torch.tensor(s.lengths, dtype=torch.int32, device="cuda")
        ltc.cache_write(s.cache, k, v, s.gtable, s.glengths)
        s.o, status = co.write(s.o, k64, v64, s.table, s.lengths)
        same_cache(s, s.o)


@pytest.mark.parametrize("codes,dtype", [("e4m3", BF), ("int8", FP)])
def test_write_extremes(ltc, codes, dtype):
    """Zeros, signed zeros, subnormals, the type's largest numbers, infinities
    and NaN; exact borders of a scale; ties."""
    s = Setup(ltc, 6, 1, 64, 16, codes, dtype, [16] * 8, [0] * 8)
    k, k64 = s.rows16(1)
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -24
    x = k.cpu().double()
    x[0:16] = 0.0
    x[16:32] = -0.0
    x[32:48] = tiny * torch.randint(-3, 4, (16, 1, 64))
    x[48:64] *= big / 8
    x[50, 0, 3], x[51, 0, 4] = big, -big
    x[64:80, 0, 5] = float("inf")
    x[65, 0, 6], x[66, 0, 7] = -float("inf"), float("nan")
    x[80:96] = float("nan")
    top = co.TOP[codes]
    x[96:112] = torch.randint(0, 33, (16, 1, 64)) / 2.0
    x[96, 0, 0] = top              # fits a scale of 1 exactly
    x[112:128] = torch.randint(0, 33, (16, 1, 64)) / 2.0
    x[112, 0, 0] = 464.0 if codes == "e4m3" else 127.5  # just past it
    k = x.to(dtype).cuda()
    k64 = x.to(dtype).double().numpy()
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    s.o, _ = co.write(s.o, k64, k64, s.table, s.lengths, s.cu)
    same_cache(s, s.o)


@pytest.mark.parametrize("case", list(SPANS))
def test_read(ltc, case):
    H, D, P, codes, dtype, new, past = SPANS[case]
    banner(f"read {case}")
    s = Setup(ltc, 12, H, D, P, codes, dtype, new, past, spread=3)
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
    wk, wv, status = co.read(s.o, s.table, s.lengths, s.cu, s.rows)
    close(k, wk, 0.0, dtype)
    close(v, wv, 0.0, dtype)
    assert int(s.cache.status.item()) == status == 0


def test_read_single_rows(ltc):
    s = Setup(ltc, 13, 3, 128, 64, "e4m3", BF, [1] * 70, [(i * 13) % 150 for i in range(70)], single=True)
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths)
    wk, wv, _ = co.read(s.o, s.table, s.lengths, None, s.rows)
    close(k, wk, 0.0, BF)
    close(v, wv, 0.0, BF)


@pytest.mark.parametrize("group", [1, 3, 16])
@pytest.mark.parametrize("case", list(SPANS))
def test_attend(ltc, case, group):
    H, D, P, codes, dtype, new, past = SPANS[case]
    banner(f"attend {case} group {group}")
    s = Setup(ltc, 14, H, D, P, codes, dtype, new, past)
    check_attend(ltc, s, H * group)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1 << 30])
@pytest.mark.parametrize("codes,dtype,dim,page", [("e4m3", BF, 128, 64), ("int8", FP, 64, 16)])
def test_attend_window(ltc, codes, dtype, dim, page, window):
    banner(f"attend window {window} {codes}")
    s = Setup(ltc, 15, 2, dim, page, codes, dtype, [1, 70, 5, 130], [300, 100, 0, 64])
    check_attend(ltc, s, 4, window)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("codes,dtype,dim,group", [("e4m3", BF, 128, 4), ("int8", FP, 96, 1), ("e4m3", FP, 256, 7),
                                                   ("int8", BF, 192, 8)])
def test_attend_single_rows(ltc, codes, dtype, dim, group, length):
    banner(f"attend one row at length {length}, dim {dim}")
    s = Setup(ltc, length, 2, dim, 32, codes, dtype, [1, 1, 1], [length - 1, length // 2, 0], single=True)
    check_attend(ltc, s, 2 * group)
    check_attend(ltc, s, 2 * group, window=40)


def test_attend_long(ltc):
    """One row over a long context, split over many workgroups."""
    s = Setup(ltc, 3, 1, 64, 64, "e4m3", BF, [1], [40000], single=True)
    check_attend(ltc, s, 2)
    s = Setup(ltc, 3, 1, 128, 128, "int8", FP, [3, 1], [20000, 10], single=False)
    check_attend(ltc, s, 4)


@pytest.mark.parametrize("new,past", [([200], [0]), ([129, 300], [700, 0]), ([64, 1, 257], [64, 500, 31])])
@pytest.mark.parametrize("codes,dtype,dim,page,heads,group", [("e4m3", BF, 128, 64, 1, 4), ("int8", FP, 64, 16, 2, 1),
                                                              ("e4m3", FP, 256, 128, 1, 5), ("int8", BF, 96, 32, 1, 7),
                                                              ("e4m3", BF, 192, 256, 1, 2)])
def test_attend_prompts(ltc, codes, dtype, dim, page, heads, group, new, past):
    banner(f"attend prompts {new} after {past}, dim {dim} group {group}")
    s = Setup(ltc, 21, heads, dim, page, codes, dtype, new, past)
    check_attend(ltc, s, heads * group)
    check_attend(ltc, s, heads * group, window=90)


@pytest.mark.parametrize("spread", [40, 90])
@pytest.mark.parametrize("new,past", [([1, 5], [300, 200]), ([140], [300])])
def test_attend_far_scales(ltc, spread, new, past):
    """Scales of neighbouring pages many powers of two apart, and pages of
    zeros at the lowest scale."""
    s = Setup(ltc, 31, 1, 64, 16, "e4m3", BF, new, past)
    sc = s.o["scales"]
    sc[:, :, 1] = s.rng.integers(127 - spread, 127 + spread // 3, sc[:, :, 1].shape)
    zero = s.rng.random(len(sc)) < 0.3
    s.o["k"][zero], s.o["v"][zero] = 0, 0
    sc[zero] = 27
    s.upload(ltc)
    check_attend(ltc, s, 3)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e3])
def test_attend_query_sizes(ltc, size):
    """Queries of zeros, of numbers far below and far above one: the softmax
    over equal scores, and over one winner."""
    for new, past in (([1, 1], [200, 5]), ([150], [10])):
        s = Setup(ltc, 32, 2, 64, 32, "int8", BF, new, past)
        check_attend(ltc, s, 4, size=size)
        check_attend(ltc, s, 4, size=size, scale=1.5)


@pytest.mark.parametrize("new,past", [([5], [100]), ([70, 1], [3, 40])])
def test_hidden_nan_does_not_count(ltc, new, past):
    """A NaN at a position is seen by the rows that see the position, and by
    no other."""
    s = Setup(ltc, 33, 1, 64, 32, "e4m3", BF, new, past)
    for t, d, which in ((past[0] + 2, 5, "v"), (past[0] + 3, 60, "v"), (0, 1, "v"), (1, 2, "k")):
        s.o[which][s.table[0, t // 32], 0, t % 32, d] = 0x7f if d % 2 else 0xff
    s.upload(ltc)
    for window in (0, 20):
        q, q64 = s.rows16(3, 1.0)
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window)
        want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu, window)
        assert np.isnan(want).any() and (window == 0 or not np.isnan(want).all())
        close(out, want, np.where(np.isnan(slack), 0.0, slack), BF)


def test_query_nan_stays_in_its_row(ltc):
    for new, past in (([1, 1, 1], [70, 80, 5]), ([150], [10])):
        s = Setup(ltc, 34, 1, 64, 32, "e4m3", FP, new, past)
        q, q64 = s.rows16(4, 1.0)
        q[0, 1, 7], q64[0, 1, 7] = float("nan"), float("nan")
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        want, slack, _ = co.attend(s.o, q64, s.table, s.lengths, s.cu)
        assert np.isnan(want).sum() == 64
        close(out, want, np.where(np.isnan(slack), 0.0, slack), FP)


def test_bad_pages_and_sequences(ltc):
    """Table entries outside the cache, lengths past the table, row offsets
    that decrease: nothing else changes, the status says so."""
    s = Setup(ltc, 41, 2, 64, 16, "e4m3", BF, [20, 5, 33, 4, 7], [30, 0, 40, 9, 3])
    s.table[0, 2] = -1
    s.table[2, 4] = len(s.o["scales"])
    s.table[2, 1] = 2 ** 31 - 1
    s.lengths[3] = s.table.shape[1] * 16 + 1
    s.lengths[4] = 6  # fewer positions than rows
    s.upload(ltc)
    q, q64 = s.rows16(4, 1.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    want, slack, status = co.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, BF)
    assert int(s.cache.status.item()) == status == 3
    with pytest.raises(ltc.LTCError):
        s.cache.check()
    s.cache.check()
    k, v = ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
    wk, wv, status = co.read(s.o, s.table, s.lengths, s.cu, s.rows)
    close(k, wk, 0.0, BF)
    close(v, wv, 0.0, BF)
    assert int(s.cache.status.item()) == status == 3
    s.cache.status.zero_()
    k, k64 = s.rows16(2)
    ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
    s.o, status = co.write(s.o, k64, k64, s.table, s.lengths, s.cu)
    same_cache(s, s.o)
    assert int(s.cache.status.item()) == status == 3


def test_bad_row_offsets(ltc):
    s = Setup(ltc, 42, 1, 64, 16, "int8", FP, [20, 5, 33, 4], [30, 0, 40, 9])
    before = {**s.o}
    for cu in ([0, 20, 10, 58, 62], [0, 20, 25, 58, 63], [-1, 20, 25, 58, 62], [0, 2 ** 31 - 1, 25, -2 ** 31, 62]):
        s.cu = np.array(cu, np.int32)
        s.upload(ltc)
        k, k64 = s.rows16(1)
        ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows)
        ltc.cache_attend(s.cache, k, s.gtable, s.glengths, s.gcu)
        assert int(s.cache.status.item()) == 2
        s.cache.status.zero_()
        ltc.cache_write(s.cache, k, k, s.gtable, s.glengths, s.gcu)
        assert int(s.cache.status.item()) == 2
        banner(f"cu {cu} refused on the device")
    assert before.keys() == s.o.keys()


def test_strides(ltc):
    """Keys, values and queries as slices of one product; a table that is a
    slice of a wider one; rows that are not 16-byte aligned."""
    for dim, off in ((128, 0), (64, 8), (64, 4)):
        s = Setup(ltc, 43, 2, dim, 32, "e4m3", BF, [40, 3, 1], [10, 31, 64])
        fused = torch.from_numpy(s.rng.normal(0, 1, (s.rows, 8 * dim + 24))).to(BF).cuda()[:, off:off + 8 * dim]
        parts = [x.unflatten(1, (-1, dim)) for x in (fused[:, :4 * dim], fused[:, 4 * dim:6 * dim], fused[:, 6 * dim:])]
        wide = torch.full((3, 2 * s.table.shape[1]), -7, dtype=torch.int32, device="cuda")
        wide[:, :s.table.shape[1]] = s.gtable
        table = wide[:, :s.table.shape[1]]
        q, k, v = parts
        ltc.cache_write(s.cache, k, v, table, s.glengths, s.gcu)
        s.o, _ = co.write(s.o, k.double().cpu().numpy(), v.double().cpu().numpy(), s.table, s.lengths, s.cu)
        same_cache(s, s.o)
        out = ltc.cache_attend(s.cache, q, table, s.glengths, s.gcu)
        want, slack, _ = co.attend(s.o, q.double().cpu().numpy(), s.table, s.lengths, s.cu)
        close(out, want, slack, BF)


def test_far_offsets(ltc):
    """Pages more than 4 GiB into the codes."""
    H, D, P = 8, 128, 64
    pages = (5 << 30) // (H * D * P)
    shape = (pages, H, P // 16)
    cache = ltc.KVCache.of(torch.empty(shape + (D // 16, 16, 16), dtype=torch.uint8, device="cuda"),
                           torch.empty(shape + (D, 16), dtype=torch.uint8, device="cuda"),
                           torch.empty((pages, H, 2), dtype=torch.uint8, device="cuda"))
    near = Setup(ltc, 44, H, D, P, "e4m3", BF, [130, 1], [0, 0], nan_behind=False)
    k, _ = near.rows16(H)
    v, _ = near.rows16(H)
    q, _ = near.rows16(H, 2.0)
    far = near.gtable.clone()
    far[0, :3] = torch.tensor([pages - 1, pages - 5, pages - 2], device="cuda")
    far[1, 0] = pages - 3
    got = []
    for c, table in ((cache, far), (near.cache, near.gtable)):
        ltc.cache_write(c, k, v, table, near.glengths, near.gcu)
        got.append((*ltc.cache_read(c, table, near.glengths, near.gcu, rows=131),
                    ltc.cache_attend(c, q, table, near.glengths, near.gcu),
                    ltc.cache_attend(c, q[:2], table, near.glengths)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    cache.check()


def test_empty_calls(ltc):
    s = Setup(ltc, 45, 2, 64, 16, "e4m3", BF, [1], [3])
    none = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    before = s.got()
    ltc.cache_write(s.cache, none, none, s.gtable, s.glengths, zero)
    assert ltc.cache_attend(s.cache, none, s.gtable, s.glengths, zero).shape == (0, 2, 64)
    assert ltc.cache_read(s.cache, s.gtable, s.glengths, zero, rows=0)[0].shape == (0, 2, 64)
    no_seq = (s.gtable[:0], s.glengths[:0])
    assert ltc.cache_attend(s.cache, none, *no_seq).shape == (0, 2, 64)
    for a, b in zip(before, s.got()):
        assert np.array_equal(a, b)
    # a sequence of length zero without rows beside one with
    s = Setup(ltc, 46, 2, 64, 16, "e4m3", BF, [0, 3], [0, 0])
    check_attend(ltc, s, 2)


@pytest.mark.parametrize("new,past", [([1, 1, 1], [300, 5, 70]), ([40, 3, 170], [10, 31, 64])])
def test_graph_and_streams(ltc, new, past):
    """A captured write and attend replayed between eager work, and the same
    on a stream of its own, give the eager results."""
    single = max(new) == 1
    s = Setup(ltc, 47, 2, 128, 64, "e4m3", BF, new, past, single=single)
    k, _ = s.rows16(2)
    v, _ = s.rows16(2)
    q, _ = s.rows16(8, 2.0)
    first = [x.clone() for x in (s.cache.k_codes, s.cache.v_codes, s.cache.scales)]

    def restore():
        for x, y in zip((s.cache.k_codes, s.cache.v_codes, s.cache.scales), first):
            x.copy_(y)

    def step():
        ltc.cache_write(s.cache, k, v, s.gtable, s.glengths, s.gcu)
        return (ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu),
                *ltc.cache_read(s.cache, s.gtable, s.glengths, s.gcu, rows=s.rows))

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    restore()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        held = step()
    for _ in range(4):
        restore()
        for x in held:
            x.fill_(7.0)
        junk = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
        torch.cuda.synchronize()
        del junk
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def test_refusals(ltc):
    s = Setup(ltc, 48, 2, 64, 16, "e4m3", BF, [4, 3], [10, 0])
    k, _ = s.rows16(2)
    args = (s.gtable, s.glengths, s.gcu)
    with pytest.raises(ValueError):
        ltc.cache_write(s.cache, k.half(), k.half(), *args)
    with pytest.raises(ValueError):
        ltc.cache_write(s.cache, k[:, :1], k[:, :1], *args)
    with pytest.raises(ValueError):
        ltc.cache_write(s.cache, k, k[:3], *args)
    with pytest.raises(ValueError):
        ltc.cache_write(s.cache, k, k, s.gtable, s.glengths)  # seven rows, two sequences
    with pytest.raises(ValueError):
        ltc.cache_attend(s.cache, k.cpu(), *args)
    with pytest.raises(ValueError):
        ltc.cache_attend(s.cache, k, s.gtable.long(), s.glengths, s.gcu)
    with pytest.raises(ValueError):
        ltc.cache_attend(s.cache, k, s.gtable[:1], s.glengths, s.gcu)
    with pytest.raises(ValueError):
        ltc.cache_attend(s.cache, k, s.gtable, s.glengths, s.gcu[:2])
    with pytest.raises(ltc.LTCError):
        ltc.cache_attend(s.cache, torch.cat([k, k[:, :1]], 1), *args)  # three query heads over two
    with pytest.raises(ltc.LTCError):
        ltc.cache_attend(s.cache, k, *args, window=-1)
    with pytest.raises(ltc.LTCError):
        ltc.cache_attend(s.cache, k, *args, scale=float("nan"))
    with pytest.raises(ValueError):
        ltc.cache_read(s.cache, *args)
    for bad in ((k.view(torch.uint8),) * 3, (s.cache.k_codes, s.cache.k_codes, s.cache.scales),
                (s.cache.k_codes, s.cache.v_codes, s.cache.scales[:1]),
                (s.cache.k_codes.cpu(), s.cache.v_codes, s.cache.scales),
                (s.cache.k_codes.transpose(4, 5), s.cache.v_codes, s.cache.scales)):
        with pytest.raises(ValueError):
            ltc.KVCache.of(*bad)
    with pytest.raises(ltc.LTCError):
        ltc.KVCache.of(s.cache.k_codes, s.cache.v_codes, s.cache.scales, dtype=torch.float32)
    with pytest.raises(ltc.LTCError):
        ltc.KVCache.of(s.cache.k_codes, s.cache.v_codes, s.cache.scales, codes="e5m2")
    s.cache.check()
