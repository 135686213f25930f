"""The operators in a row, as a served layer uses them: the example runs, and a
run of rotation, write, weighed attention and eviction against 64 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import cache4_oracle as c4
import evict_oracle as eo
from cache4_setup import Setup4, close
from test_gpu_rotate import oracle as rotate_oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("codes", ["e2m1", "e4m3", "int8"])
def test_example(ltc, codes):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_bounded
    cuts, held, total, worst = serve_bounded.main(steps=150, codes=codes)
    assert cuts == 3 and total == [550, 240, 407]
    assert held[0] == held[2] == 192 + 150 - 2 * 64 and held[1] <= 192 + 64
    # a last row: values up to 6 in 16 bits, rounded once as they are read and once as output, and weights of 16 bits
    assert worst < 6 * (2 * 2.0 ** -8 + 2.0 ** -10)


def test_a_run_of_them(ltc):
    """Prompts of two sequences, decoding, a cut, decoding again: codes, positions
    and new lengths equal to the oracle's, rows and weights within its slack."""
    H, G, D, P, keep, recent = 2, 2, 64, 16, 40, 6
    s = Setup4(ltc, 91, H, D, P, BF, [50, 23], [0, 0], spare=12)
    rot = ltc.Rotation(D)
    rates = [10000.0 ** (-2.0 * i / D) for i in range(D // 2)]
    w = s.cache.no_weights()
    want_w, slack_w = np.zeros(tuple(w.shape)), np.zeros(tuple(w.shape))
    w1 = torch.ones(D, dtype=BF, device="cuda")
    total, rng = list(s.lengths), s.rng

    def pass_(new):
        nonlocal want_w, slack_w
        rows = sum(new)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q, k, v = (torch.from_numpy(rng.normal(0, 1, (rows, h, D))).to(BF).cuda() for h in (H * G, H, H))
        gpu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (total, s.lengths)]
        gcu, table = torch.from_numpy(cu).cuda(), torch.from_numpy(s.table).cuda()
        a, b = ltc.norm_rotate(q, k, rot, gpu[0], gcu, w1, w1)
        positions = [n - m + i for n, m in zip(total, new) for i in range(m)]
        for x, y in ((q, a), (k, b)):
            want, size = rotate_oracle(x.double().cpu().numpy(), positions, rates, D, False, np.ones(D), 1e-6)
            off = np.abs(y.double().cpu().numpy() - want)
            assert (off <= 2.0 ** -19 * size + 2.0 ** -8 * (np.abs(want) + 2.0 ** -19 * size)).all()
        ltc.cache_write(s.cache, b, v, table, gpu[1], gcu)
        s.o, status = c4.write(s.o, b.double().cpu().numpy(), v.double().cpu().numpy(), s.table, s.lengths, cu)
        s.same(s.o)
        out = ltc.cache_attend(s.cache, a, table, gpu[1], gcu, weights=w)
        want, slack, shares, off, status2 = eo.attend(s.o, a.double().cpu().numpy(), s.table, s.lengths, cu)
        close(out, want, slack, BF)
        before = slack_w
        want_w, more = eo.weigh(s.o, want_w, shares, off, s.table, s.lengths, cu, rows)
        slack_w = before + more
        assert (np.abs(w.double().cpu().numpy() - want_w) <= slack_w).all() and status == status2 == 0

    pass_([50, 23])
    for _ in range(4):
        s.lengths = [n + 1 for n in s.lengths]
        total = [n + 1 for n in total]
        pass_([1, 1])
    # the pages of the cut, and the rest of a table that grows into further ones
    used = {int(p) for i, n in enumerate(s.lengths) for p in s.table[i, :-(-n // P)]}
    free = [p for p in range(s.pages) if p not in used]
    to = np.array(free[:8], np.int32).reshape(2, 4)
    held = w.cpu().numpy()
    lengths, positions = ltc.cache_evict(s.cache, w, torch.from_numpy(s.table).cuda(),
                                         torch.tensor(s.lengths, dtype=torch.int32, device="cuda"), torch.from_numpy(to).cuda(), keep, recent)
    s.o, want_h, n, want_p, status = eo.evict(s.o, held, s.table, s.lengths, to, keep, recent)
    assert lengths.tolist() == n == [40, 27] and np.array_equal(positions.cpu().numpy(), want_p) and status == 0
    s.same(s.o)
    assert np.array_equal(w.cpu().numpy(), want_h)
    want_w, slack_w = want_h.astype(np.float64), np.zeros_like(slack_w)
    s.table, s.lengths = to, n
    for _ in range(3):
        s.lengths = [m + 1 for m in s.lengths]
        total = [m + 1 for m in total]
        pass_([1, 1])
    assert total == [57, 30] and s.lengths == [43, 30]
    assert int(s.cache.status.item()) == 0
