"""Attention over the 8-bit cache where one position takes nearly all of the
weight and its own values are zero: the output is what thousands of weights
far below it make of their values.  The bound on the error does not grow with
the number of positions."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, HALF, ltc  # noqa: F401

pytestmark = pytest.mark.gpu

HEAD = 9       # a weight is 2^HEAD times its share of the largest when it is rounded to fp16
SPREAD = 0.5   # the other scores' distance from zero, nats

# query heads a key head, rows and positions of each sequence, sequences; heads * tiles decide which kernel runs
CALLS = {
    "tiles": (16, 120, (8220, 8117), True),
    "rows": (16, 1, tuple(8192 + i for i in range(32)), False),
    "rows, two column blocks": (2, 16, tuple(8192 + i for i in range(32)), True),
    "rows, split": (8, 1, (8200,), False),
}


class Sink:
    """One run of pages that every sequence of the call looks at.  Scores are
    query number 0 times key number 0, which only the sink has, plus number 1,
    which is within SPREAD for every key."""

    def __init__(self, ltc, codes, dtype, length, sink, far, heads=16, dim=64, page=64, seed=0):  # noqa: F811
        rng = np.random.default_rng(seed)
        pages = -(-length // page)
        shape = (pages, heads, page, dim)
        k, v = np.zeros(shape), np.zeros(shape)
        k[..., 1] = rng.integers(-8, 9, shape[:3]) / 16 if codes == "e4m3" else rng.integers(-1, 2, shape[:3])
        self.q1 = 1.0 if codes == "e4m3" else SPREAD
        v[:] = rng.integers(8, 16, shape) / 8 if codes == "e4m3" else rng.integers(64, 128, shape)
        k[sink // page, :, sink % page, 0] = 1.0
        k[sink // page, :, sink % page, 1] = 0.0
        v[sink // page, :, sink % page] = 0.0
        scales = np.full((pages, heads, 2), 127, np.uint8)
        scales[..., 1] -= 6
        scales[sink // page, :, 1] += far
        self.k = k.swapaxes(1, 2).reshape(-1, heads, dim)
        self.v = (v * 2.0 ** (scales[:, :, None, 1:].astype(float) - 127)).swapaxes(1, 2).reshape(-1, heads, dim)
        ks, vs = co.to_stored(co.code(k, codes), co.code(v, codes))
        self.cache = ltc.KVCache.of(torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda(),
                                    torch.from_numpy(scales).cuda(), dtype=dtype, codes=codes)
        self.pages, self.heads, self.dim = pages, heads, dim

    def want(self, q, positions):
        """softmax(q k^T) v in 64 bits of rows at these positions."""
        out = np.zeros(q.shape)
        group = q.shape[1] // self.heads
        for h in range(self.heads):
            s = q[:, h * group:(h + 1) * group] @ self.k[:, h].T
            s[np.arange(len(self.k)) > positions[:, None, None].repeat(group, 1)] = -np.inf
            p = np.exp(s - s.max(-1, keepdims=True))
            out[:, h * group:(h + 1) * group] = p @ self.v[:, h] / p.sum(-1, keepdims=True)
        return out


@pytest.mark.parametrize("gap,far", [(16, 0), (18, 0), (17, 1)])
@pytest.mark.parametrize("codes,dtype", [("e4m3", BF), ("int8", FP)])
@pytest.mark.parametrize("call", list(CALLS))
def test_sink(ltc, call, codes, dtype, gap, far):  # noqa: F811
    banner(f"sink {call} {codes} {gap} nats, its page's values times 2^{far}")
    group, rows, lengths, ragged = CALLS[call]
    s = Sink(ltc, codes, dtype, max(lengths), 5 if gap == 18 else 3001, far)
    n, heads = rows * len(lengths), s.heads * group
    q = torch.zeros((n, heads, s.dim), dtype=dtype)
    q[..., 0], q[..., 1] = gap, s.q1
    table = torch.arange(s.pages, dtype=torch.int32, device="cuda").repeat(len(lengths), 1)
    glengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda") if ragged else None
    got = ltc.cache_attend(s.cache, q.cuda(), table, glengths, cu, scale=1.0).double().cpu().numpy()
    s.cache.check()
    pick = np.arange(0, n, 7)  # the rows that are compared
    positions = np.array([lengths[i // rows] - rows + i % rows for i in pick])
    want = s.want(q[pick].double().numpy(), positions)
    # the least weight is 2^-bits of the largest: rounded to fp16 it is off by 2^-11 of itself, or by 2^-25; all
    # products are positive, so their sum is off by as much at most.  2^-10 for scores and sums in 32 bits: 8,200
    # positions in 257 sums of 32, twice, and 72 roundings of scores up to 18.
    bits = (gap + SPREAD) / np.log(2) + far
    off = max(2.0 ** -11, 2.0 ** (bits - HEAD - 25)) + 2.0 ** -10
    bad = np.abs(got[pick] - want) > want * (off + HALF[dtype] * (1 + off))
    assert (want > 0).all() and not bad.any(), (float(np.abs(got[pick] / want - 1).max()), off)
    # the rows that were not compared are the same query at neighbouring positions
    assert (np.abs(got / got[0, 0, 0] - 1) < 1).all()
