"""What each cached position is worth to a call's rows (cache_attend with
weights) against 64 bits, for each code type."""
import numpy as np
import pytest
import torch

import evict_oracle as eo
from cache4_setup import Setup4, close
from gpu_util import banner
from test_gpu_cache import Setup

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def setup(ltc, seed, heads, dim, page, codes, dtype, new, past, **kw):
    if codes == "e2m1":
        return Setup4(ltc, seed, heads, dim, page, dtype, new, past, **kw)
    return Setup(ltc, seed, heads, dim, page, codes, dtype, new, past, **kw)


def check(ltc, s, q_heads, window=0, scale=None, size=2.0, calls=1):
    weights = torch.from_numpy(s.rng.exponential(1.0, s.cache.no_weights().shape).astype(np.float32)).cuda()
    want_w = weights.double().cpu().numpy()
    total = 0.0
    for _ in range(calls):
        q, q64 = s.rows16(q_heads, size)
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, scale=scale, weights=weights)
        plain = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, scale=scale)
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
        want, slack, shares, off, status = eo.attend(s.o, q64, s.table, s.lengths, s.cu, window, scale)
        close(out, want, slack, s.dtype)
        want_w, slack_w = eo.weigh(s.o, want_w, shares, off, s.table, s.lengths, s.cu, s.rows)
        total = total + slack_w
        got = weights.double().cpu().numpy()
        bad = np.abs(got - want_w) > total
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want_w[bad][:5], total[bad][:5])
    assert int(s.cache.status.item()) == status == 0


TYPES = [("e4m3", BF), ("int8", FP), ("e2m1", BF), ("e4m3", FP), ("int8", BF), ("e2m1", FP)]
# heads, dim, page, new rows, positions before them
SPANS = {
    "one token": (2, 64, 16, [1, 1, 1], [0, 16, 32]),
    "ragged": (2, 128, 64, [1, 17, 64, 65, 130, 3], [0, 5, 0, 63, 64, 200]),
    "no rows": (1, 192, 128, [0, 5, 0, 0, 129, 0], [7, 3, 0, 128, 127, 1]),
    "large heads": (1, 256, 256, [300, 2], [5, 254]),
    "odd heads": (7, 96, 64, [70, 1, 9], [3, 77, 0]),
}


@pytest.mark.parametrize("codes,dtype", TYPES)
@pytest.mark.parametrize("case", list(SPANS))
def test_weigh(ltc, case, codes, dtype):
    H, D, P, new, past = SPANS[case]
    banner(f"weigh {case} {codes}")
    check(ltc, setup(ltc, 51, H, D, P, codes, dtype, new, past), 3 * H)


@pytest.mark.parametrize("window", [1, 17, 64, 65, 200])
@pytest.mark.parametrize("codes,dtype", TYPES[:3])
def test_window(ltc, codes, dtype, window):
    check(ltc, setup(ltc, 52, 2, 128, 32, codes, dtype, [1, 70, 5, 130], [300, 100, 0, 64]), 4, window)


@pytest.mark.parametrize("window", [1, 16, 63, 100, 5000])
@pytest.mark.parametrize("codes,dtype,dim,page", [("e4m3", BF, 128, 16), ("int8", FP, 64, 64), ("e2m1", BF, 96, 32), ("e2m1", FP, 256, 16)])
def test_window_of_few_rows(ltc, codes, dtype, dim, page, window):
    """Rows few enough for their scores to be written down."""
    check(ltc, setup(ltc, 63, 2, dim, page, codes, dtype, [1, 4, 0, 2, 5], [300, 1100, 17, 0, 64]), 6, window)
    check(ltc, setup(ltc, 64, 2, dim, page, codes, dtype, [1, 1, 1], [2047, 0, 64], single=True), 2, window)


@pytest.mark.parametrize("codes,dtype", TYPES[:3])
def test_single_rows_again_and_again(ltc, codes, dtype):
    """Without row offsets; calls add up, but for the row's own position."""
    check(ltc, setup(ltc, 53, 3, 128, 64, codes, dtype, [1] * 20, [(i * 41) % 500 for i in range(20)], single=True), 12, calls=3)


@pytest.mark.parametrize("codes,dtype", TYPES[:3])
def test_long_row(ltc, codes, dtype):
    """Split over many workgroups, both passes."""
    check(ltc, setup(ltc, 54, 1, 64, 64, codes, dtype, [1], [30001], single=True), 4)


@pytest.mark.parametrize("codes,dtype", TYPES[:3])
def test_shared_positions_kernel(ltc, codes, dtype):
    """Enough rows and heads for the attention kernel whose waves share positions."""
    check(ltc, setup(ltc, 55, 8, 64, 32, codes, dtype, [300, 9, 300] + [64] * 8, [100, 0, 3] + [5] * 8), 64)


@pytest.mark.parametrize("codes,dtype", TYPES[:3])
@pytest.mark.parametrize("size", [0.0, 60.0])
def test_sizes_of_scores(ltc, codes, dtype, size):
    """Equal scores, and one winner a row."""
    check(ltc, setup(ltc, 56, 2, 64, 16, codes, dtype, [5, 1, 40], [100, 33, 2]), 4, size=size)


def test_far_value_scales(ltc):
    """Value scales say nothing about weights, however far apart."""
    s = Setup4(ltc, 57, 1, 64, 16, BF, [1, 5, 140], [300, 200, 20])
    s.o["ve"][:] = s.rng.integers(27, 160, s.o["ve"].shape)
    s.upload(ltc)
    check(ltc, s, 3)


def test_rows_add_up_to_their_number(ltc):
    """Weights of all positions: one for each row and query head."""
    s = Setup4(ltc, 58, 4, 128, 64, BF, [500, 3], [70, 1000])
    w = s.cache.no_weights()
    ltc.cache_attend(s.cache, s.rows16(8)[0], s.gtable, s.glengths, s.gcu, weights=w)
    # 4 heads, 2 query heads each; a sum of 571,000 numbers at most 1 off by 2^-22 of itself each
    assert abs(float(w.double().sum()) - 503 * 8) < 503 * 8 * 2.0 ** -14


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_nan_reaches_what_its_row_sees(ltc, codes):
    s = setup(ltc, 59, 1, 64, 32, codes, BF, [5, 2], [100, 40])
    w = s.cache.no_weights()
    q = s.rows16(4)[0]
    q[2, 1, 7] = float("nan")
    ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, weights=w)
    nan = torch.isnan(w).cpu().numpy()
    for i, (n, bad) in enumerate(((105, 103), (42, 0))):
        for t in range(n):
            assert nan[s.table[i, t // 32], 0, t % 32] == (t < bad)


@pytest.mark.parametrize("new,past", [([20, 5, 33, 4, 7], [30, 0, 40, 9, 3]), ([1, 5, 3, 4, 7], [40, 0, 75, 9, 3])])
def test_bad_pages_and_sequences(ltc, new, past):
    s = Setup4(ltc, 60, 2, 64, 16, BF, new, past)
    s.table[0, 2] = -1
    s.table[2, 4] = s.pages
    s.lengths[3] = s.table.shape[1] * 16 + 1
    s.lengths[4] = 6
    s.upload(ltc)
    w = torch.from_numpy(s.rng.exponential(1.0, (s.pages, 2, 16)).astype(np.float32)).cuda()
    before = w.double().cpu().numpy()
    q, q64 = s.rows16(4, 1.0)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, weights=w)
    want, slack, shares, off, status = eo.attend(s.o, q64, s.table, s.lengths, s.cu)
    close(out, want, slack, BF)
    want_w, slack_w = eo.weigh(s.o, before, shares, off, s.table, s.lengths, s.cu, s.rows)
    assert (np.abs(w.double().cpu().numpy() - want_w) <= slack_w).all()
    assert int(s.cache.status.item()) == status == 3


def test_captured(ltc):
    """Replays of a captured call add up as calls do, with eager calls between them."""
    s = Setup4(ltc, 61, 2, 128, 32, BF, [1] * 5, [600, 5, 70, 1000, 31], single=True)
    q = s.rows16(8)[0]
    a, b = s.cache.no_weights(), s.cache.no_weights()
    ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=s.cache.no_weights())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=a)
    for i in range(4):
        q.copy_(s.rows16(8)[0])
        graph.replay()
        want = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=b)
        assert torch.equal(out, want) and torch.equal(a, b) and float(a.sum()) > 0
        torch.cuda.synchronize()


def test_two_streams_and_two_caches(ltc):
    """Calls at once on two streams, each with workspaces of its own."""
    a = Setup4(ltc, 65, 2, 128, 32, BF, [1] * 5, [600, 5, 70, 1000, 31], single=True)
    q = [a.rows16(8)[0] for _ in range(2)]
    w = [a.cache.no_weights() for _ in range(2)]
    want = [ltc.cache_attend(a.cache, q[i], a.gtable, a.glengths, weights=w[i]) for i in range(2)]
    want_w = [x.clone() for x in w]
    for x in w:
        x.zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                w[i].zero_()
                got.append(ltc.cache_attend(a.cache, q[i], a.gtable, a.glengths, weights=w[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))
    assert all(torch.equal(x, y) for x, y in zip(w, want_w))


def test_refusals(ltc):
    s = Setup4(ltc, 62, 2, 64, 16, BF, [1], [5], single=True)
    q, w = s.rows16(2)[0], s.cache.no_weights()
    for bad in (w.half(), w[:1], w.cpu(), w.transpose(0, 1).contiguous().transpose(0, 1), w.clone().requires_grad_()):
        with pytest.raises(ValueError):
            ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=bad)
    assert not w.any()
