"""Positions outside the windows of a call's rows: their weights are not
touched, so their pages may be another sequence's of the same call."""
import numpy as np
import pytest
import torch

import evict_oracle as eo
from cache4_setup import close
from gpu_util import banner
from test_gpu_cache_weigh import BF, FP, check, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("window", [1, 16, 37, 100, 640])
@pytest.mark.parametrize("codes,dtype,new,past", [("e2m1", BF, [1, 3, 2], [1500, 900, 700]), ("int8", FP, [1, 3, 2], [1500, 900, 700]),
                                                  ("e4m3", BF, [130, 90, 300], [1500, 900, 700]), ("e2m1", FP, [30, 9, 40], [1500, 900, 700])])
def test_pages_behind_the_window_are_another_sequence_s(ltc, codes, dtype, new, past, window):
    """Every entry of a sequence's table that lies before its first row's window
    names a page of the next sequence, one that its rows see."""
    banner(f"weigh {codes} {new}, window {window}, stale entries")
    s = setup(ltc, 82, 2, 64, 16, codes, dtype, new, past)
    own = s.table.copy()
    seen = [((n + p - 1) // 16, max(p + 1 - window, 0) // 16) for n, p in zip(new, past)]
    for i in range(3):
        last, first = seen[(i + 1) % 3]
        for j in range(seen[i][1]):
            s.table[i, j] = own[(i + 1) % 3, last - j % (last - first + 1)]
    assert all(first >= 3 for _, first in seen)
    s.gtable = torch.from_numpy(s.table).cuda()
    w = torch.from_numpy(s.rng.exponential(1.0, tuple(s.cache.no_weights().shape)).astype(np.float32)).cuda()
    before = w.double().cpu().numpy()
    q, q64 = s.rows16(6)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, weights=w)
    want, slack, shares, off, status = eo.attend(s.o, q64, s.table, s.lengths, s.cu, window)
    close(out, want, slack, dtype)
    # the definition, but for positions that no row sees: those keep what they have
    want_w, slack_w, looked = before.copy(), np.zeros(before.shape), np.zeros(before.shape, bool)
    for i, (n, p) in enumerate(zip(new, past)):
        for t in range(max(p + 1 - window, 0), n + p):
            page, at = s.table[i, t // 16], t % 16
            assert not looked[page, :, at].any()
            looked[page, :, at] = True
            want_w[page, :, at] = (before[page, :, at] if t < p else 0.0) + shares[i][:, t]
            slack_w[page, :, at] = off[i][:, t] + 2.0 ** -24 * np.abs(want_w[page, :, at])
    got = w.double().cpu().numpy()
    assert np.array_equal(got[~looked], before[~looked])
    assert (np.abs(got - want_w) <= slack_w).all()
    assert int(s.cache.status.item()) == status == 0


@pytest.mark.parametrize("codes,dtype,new,past", [("e2m1", BF, [1, 3, 2], [1500, 900, 700]), ("e4m3", BF, [130, 90, 300], [1500, 900, 700]),
                                                  ("int8", FP, [30, 9, 40], [1500, 900, 700])])
def test_a_window_wider_than_all_positions_is_none(ltc, codes, dtype, new, past):
    """The widest that there are: the same numbers as without one."""
    s = setup(ltc, 83, 2, 64, 16, codes, dtype, new, past)
    q, _ = s.rows16(6)
    want = s.cache.no_weights()
    plain = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, weights=want)
    for window in (2 ** 31 - 1, 2 ** 31 - 64, 1 << 30):
        w = s.cache.no_weights()
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, weights=w)
        assert torch.equal(out, plain) and torch.equal(w, want) and float(w.sum()) > 0


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1024])
@pytest.mark.parametrize("codes,dtype,dim", [("e2m1", BF, 128), ("int8", FP, 64), ("e4m3", BF, 96)])
def test_scores_of_wide_tables(ltc, codes, dtype, dim, window):
    """Tables of far more positions than the windows: rows' scores begin with what the sequence's first row sees."""
    s = setup(ltc, 84, 2, dim, 16, codes, dtype, [1, 4, 0, 2, 5, 1], [4000, 1100, 17, 0, 64, 63])
    table = s.rng.integers(-5, s.pages + 5 if codes == "e2m1" else 5, (6, 9000)).astype(np.int32)
    table[:, :s.table.shape[1]] = s.table
    s.table, s.gtable = table, torch.from_numpy(table).cuda()
    check(ltc, s, 6, window)


def test_positions_that_came_without_weights(ltc):
    """What their page's earlier tokens left counts, unless it is cleared."""
    s = setup(ltc, 85, 2, 64, 16, "e4m3", BF, [1, 1], [60, 33], single=True)
    q, _ = s.rows16(4)
    alone = s.cache.no_weights()
    ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=alone)
    stale = torch.full_like(alone, 2.0)
    ltc.cache_attend(s.cache, q, s.gtable, s.glengths, weights=stale)
    for i, n in enumerate((61, 34)):
        for t in range(n):
            at = int(s.table[i, t // 16]), slice(None), t % 16
            assert torch.equal(stale[at], alone[at] + (2.0 if t < n - 1 else 0.0))
