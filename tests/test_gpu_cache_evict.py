"""Eviction by weight against its definition: which positions are kept, in
which order, and every code, scale and weight of the pages they move to."""
import numpy as np
import pytest
import torch

import evict_oracle as eo
from gpu_util import banner
from test_gpu_cache import same_cache
from test_gpu_cache_weigh import BF, FP, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def prepared(ltc, seed, heads, dim, page, codes, dtype, lengths, keep, weights=None):
    """A cache with pages for the kept positions besides those in use, and weights."""
    kept = -(-keep // page)
    spare = kept * len(lengths)
    past = [n - 1 for n in lengths]
    if codes == "e2m1":
        s = setup(ltc, seed, heads, dim, page, codes, dtype, [1] * len(lengths), past, single=True, spare=spare)
        free = s.free
    else:
        # spare pages: those of further sequences, which the call does not name
        s = setup(ltc, seed, heads, dim, page, codes, dtype, [1] * (len(lengths) + spare), past + [page - 1] * spare, single=True)
        free = s.table[len(lengths):, 0]
        s.table, s.lengths, s.rows = s.table[:len(lengths)], s.lengths[:len(lengths)], len(lengths)
        s.gtable, s.glengths = s.gtable[:len(lengths)], s.glengths[:len(lengths)]
    s.to = free[:spare].reshape(len(lengths), kept).astype(np.int32)
    shape = tuple(s.cache.no_weights().shape)
    s.w = s.rng.exponential(1.0, shape).astype(np.float32) if weights is None else weights(s.rng, shape)
    return s


def check(ltc, s, keep, recent):
    w, to = torch.from_numpy(s.w.copy()).cuda(), torch.from_numpy(s.to).cuda()
    lengths, positions = ltc.cache_evict(s.cache, w, s.gtable, s.glengths, to, keep, recent)
    want, want_w, want_n, want_p, status = eo.evict(s.o, s.w, s.table, s.lengths, s.to, keep, recent)
    assert lengths.tolist() == want_n
    assert np.array_equal(positions.cpu().numpy(), want_p), np.argwhere(positions.cpu().numpy() != want_p)[:5]
    s.o = want
    if "ke" in want:
        s.same(want)
    else:
        same_cache(s, want)
    assert np.array_equal(w.cpu().numpy(), want_w, equal_nan=True)
    assert int(s.cache.status.item()) == status
    return lengths, w


CASES = {  # heads, dim, page, lengths, keep, recent
    "ragged": (2, 64, 16, [1, 15, 16, 17, 40, 100, 33], 20, 4),
    "nothing recent": (3, 128, 32, [200, 77, 64], 33, 0),
    "only recent": (1, 96, 64, [130, 64, 300], 65, 65),
    "one kept": (2, 64, 16, [50, 1, 2], 1, 0),
    "one kept, the last": (2, 64, 16, [50, 1, 2], 1, 1),
    "keep is the length": (1, 192, 32, [96, 95, 97], 96, 5),
    "large heads": (1, 256, 256, [700, 255], 300, 10),
    "long": (2, 64, 64, [5000, 2049, 1024], 1025, 100),
    "nearly all": (1, 128, 64, [3001], 3000, 1),
}


@pytest.mark.parametrize("codes,dtype", [("e2m1", BF), ("e4m3", BF), ("int8", FP)])
@pytest.mark.parametrize("case", list(CASES))
def test_evict(ltc, case, codes, dtype):
    H, D, P, lengths, keep, recent = CASES[case]
    banner(f"evict {case} {codes}")
    check(ltc, prepared(ltc, 71, H, D, P, codes, dtype, lengths, keep), keep, recent)


def _ties(rng, shape):
    return rng.integers(0, 4, shape).astype(np.float32)


def _odd(rng, shape):
    """Infinities, NaN, zeros of both signs, negative and subnormal numbers."""
    x = rng.choice(np.array([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, -1.5, 1e-45, -1e-45, 2.0, 3e38], np.float32), shape)
    return np.where(rng.random(shape) < 0.3, rng.normal(0, 1, shape).astype(np.float32), x)


@pytest.mark.parametrize("codes,dtype", [("e2m1", FP), ("int8", BF)])
@pytest.mark.parametrize("weights", [_ties, _odd, lambda rng, shape: np.zeros(shape, np.float32),
                                     lambda rng, shape: np.full(shape, np.nan, np.float32)])
@pytest.mark.parametrize("keep,recent", [(40, 0), (100, 17), (131, 64)])
def test_ties_and_odd_weights(ltc, weights, codes, dtype, keep, recent):
    check(ltc, prepared(ltc, 72, 2, 64, 32, codes, dtype, [150, 1200, 90, 2500], keep, weights), keep, recent)


def _few_hundreds(rng, shape):
    return (rng.integers(0, 300, shape) / 300).astype(np.float32)


@pytest.mark.parametrize("weights", [None, _ties, _odd, _few_hundreds, lambda rng, shape: np.ones(shape, np.float32)])
@pytest.mark.parametrize("heads,lengths,keep,recent", [(2, [20001, 300, 8193, 1], 5000, 40), (1, [40000], 39999, 0),
                                                       (3, [12345, 9000], 1, 0), (1, [33000], 700, 700), (1, [66000], 9000, 5)])
def test_many_positions(ltc, heads, lengths, keep, recent, weights):
    """Shared by several workgroups a sequence and head."""
    banner(f"evict {lengths} to {keep}")
    check(ltc, prepared(ltc, 79, heads, 64, 64, "e2m1", BF, lengths, keep, weights), keep, recent)


@pytest.mark.parametrize("weights", [None, _few_hundreds])
def test_many_positions_of_many_heads(ltc, weights):
    """One workgroup a sequence and head, more positions than it holds."""
    check(ltc, prepared(ltc, 80, 5, 64, 256, "int8", FP, [34000] + [1000 + 700 * i for i in range(13)], 2000, weights), 2000, 77)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_scales_far_apart(ltc, codes):
    """8-bit pages of very different scales: codes are rounded to the largest one's."""
    s = prepared(ltc, 73, 2, 64, 16, codes, BF, [150, 90], 70)
    s.o["scales"][:] = s.rng.integers(27, 200, s.o["scales"].shape)
    s.upload(ltc)
    s.gtable, s.glengths = torch.from_numpy(s.table).cuda(), torch.tensor(s.lengths, dtype=torch.int32, device="cuda")
    check(ltc, s, 70, 8)


@pytest.mark.parametrize("codes", ["e2m1", "e4m3"])
def test_the_cache_s_first_page(ltc, codes):
    """Page 0 in the middle of a sequence, its first kept token the second of 16."""
    s = prepared(ltc, 78, 2, 64, 16, codes, BF, [64], 48, lambda rng, shape: np.ones(shape, np.float32))
    swap = {0: s.table[0, 1], s.table[0, 1]: 0}
    s.table = np.vectorize(lambda p: swap.get(p, p))(s.table).astype(np.int32)
    s.to = np.vectorize(lambda p: swap.get(p, p))(s.to).astype(np.int32)
    s.gtable = torch.from_numpy(s.table).cuda()
    s.w[s.table[0, 0], :, :15] = 0.0  # position 15, then all of page 0
    check(ltc, s, 48, 0)


@pytest.mark.parametrize("codes", ["e2m1", "int8"])
def test_bad_pages_and_sequences(ltc, codes):
    s = prepared(ltc, 74, 2, 64, 16, codes, BF, [150, 90, 40, 60, 100], 70)
    s.table[0, 2], s.table[0, 9] = -1, 10 ** 6
    s.lengths[2], s.lengths[3] = s.table.shape[1] * 16 + 1, -1
    s.to[1, 1] = -7
    s.to[4, 0] = 10 ** 6
    s.gtable, s.glengths = torch.from_numpy(s.table).cuda(), torch.tensor(s.lengths, dtype=torch.int32, device="cuda")
    check(ltc, s, 70, 8)
    with pytest.raises(ltc.LTCError):
        s.cache.check()


@pytest.mark.parametrize("codes", ["e2m1", "e4m3"])
def test_a_cut_sequence_goes_on(ltc, codes):
    """Attention over the kept positions is attention over those alone, head by head."""
    s = prepared(ltc, 75, 2, 128, 32, codes, BF, [300, 77, 500], 96)
    check(ltc, s, 96, 16)
    s.table, s.lengths = s.to, [96, 77, 96]
    s.gtable = torch.from_numpy(s.to).cuda()
    s.glengths = torch.tensor(s.lengths, dtype=torch.int32, device="cuda")
    q, q64 = s.rows16(8)
    from cache4_setup import close
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths)
    want, slack, _, _, _ = eo.attend(s.o, q64, s.table, s.lengths)
    close(out, want, slack, BF)


def test_captured(ltc):
    s = prepared(ltc, 76, 2, 64, 16, "e2m1", BF, [150, 90, 600], 70)
    to = torch.from_numpy(s.to).cuda()
    w = torch.from_numpy(s.w).cuda()
    ltc.cache_evict(s.cache, w.clone(), s.gtable, s.glengths, to, 70, 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lengths, positions = ltc.cache_evict(s.cache, w, s.gtable, s.glengths, to, 70, 8)
    for i in range(4):
        w.copy_(torch.rand_like(w))
        s.w = w.cpu().numpy()
        graph.replay()
        want, want_w, want_n, want_p, _ = eo.evict(s.o, s.w, s.table, s.lengths, s.to, 70, 8)
        assert lengths.tolist() == want_n and np.array_equal(positions.cpu().numpy(), want_p)
        s.same(want)
        assert np.array_equal(w.cpu().numpy(), want_w)
        torch.cuda.synchronize()


def test_refusals(ltc):
    s = prepared(ltc, 77, 2, 64, 16, "e2m1", BF, [50, 20], 20)
    w, to = torch.from_numpy(s.w).cuda(), torch.from_numpy(s.to).cuda()
    for keep, recent in ((0, 0), (20, 21), (20, -1), (-3, 0), (2 ** 32 + 20, 0)):
        with pytest.raises(ltc.LTCError):
            ltc.cache_evict(s.cache, w, s.gtable, s.glengths, to, keep, recent)
    for bad in (to[:, :1], to.long(), to[:1], to.cpu(), to.t().contiguous().t(), to[:1].expand(2, -1)):
        with pytest.raises(ValueError):
            ltc.cache_evict(s.cache, w, s.gtable, s.glengths, bad, 20, 0)
    with pytest.raises(ValueError):
        ltc.cache_evict(s.cache, w[:-1], s.gtable, s.glengths, to, 20, 0)
    empty = ltc.cache_evict(s.cache, w, s.gtable[:0], s.glengths[:0], to[:0], 20, 0)
    assert empty[0].shape == (0,) and empty[1].shape == (0, 2, 20)
    assert np.array_equal(w.cpu().numpy(), s.w)
