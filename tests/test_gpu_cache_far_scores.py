"""Scores so large that fp32 has only whole or coarser steps for them: the
weights stay finite, and the outputs are what the distances of the scores say.
All products are powers of two times small whole numbers, so every score is
exact, and the distances are so large, or zero, that weights are 0 or 1."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, HALF, ltc  # noqa: F401

pytestmark = pytest.mark.gpu

CALLS = {"tiles": (16, 120, (220, 137), True), "rows": (16, 1, tuple(100 + i for i in range(32)), False),
         "split": (4, 1, (2000,), False), "few": (4, 5, (300, 70), True)}


def attend(ltc, call, codes, dtype, power, key, sign, seed, spread=0):  # noqa: F811
    """Outputs of queries sign * 2^power / 8 (their scale included) in dim 0 and
    1 in dim 1; key(position's share of the positions) gives the keys' first two
    numbers.  Also the values, and each row's number of positions."""
    group, rows, lengths, ragged = CALLS[call]
    heads, dim, page = 16, 64, 16
    rng = np.random.default_rng(seed)
    pages = -(-max(lengths) // page)
    shape = (pages, heads, page, dim)
    k, v = np.zeros(shape), rng.integers(64, 128, shape).astype(float)
    if codes == "e4m3":
        v = np.floor(v / 8) * 8  # four bits
    k[..., 0], k[..., 1] = (x.reshape(pages, 1, page) for x in key(np.arange(pages * page) / (pages * page)))
    scales = np.full((pages, heads, 2), 127, np.uint8)
    scales[..., 1] = 122 + rng.integers(-spread, spread + 1, (pages, heads))
    ks, vs = co.to_stored(co.code(k, codes), co.code(v, codes))
    cache = ltc.KVCache.of(*(torch.from_numpy(x).cuda() for x in (ks, vs, scales)), dtype=dtype, codes=codes)
    n = rows * len(lengths)
    scale = 2.0 ** (power - 3 - min(power - 3, 8))
    q = torch.zeros((n, heads * group, dim), dtype=dtype)
    q[..., 0], q[..., 1] = sign * 2.0 ** (power - 3) / scale, 1 / scale
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(len(lengths), 1)
    glengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda") if ragged else None
    got = ltc.cache_attend(cache, q.cuda(), table, glengths, cu, scale=scale).double().cpu().numpy()
    cache.check()
    v *= 2.0 ** (scales[:, :, None, 1:].astype(float) - 127)
    return got, v.swapaxes(1, 2).reshape(-1, heads, dim).repeat(group, 1), [
        lengths[i // rows] - rows + i % rows + 1 for i in range(n)]


def rounding(largest):
    """For scores up to `largest` (nats).  2^9 times a best weight is rounded to
    fp16; it lies below 2^9 by the bound's margin, 2^-21 of it, and two roundings
    of the exponent, each to 2^-23 of it: off by 2^-11 of itself, or by 2^-25.
    2^-10 for sums of 2,000 in 32 bits."""
    largest *= np.log2(np.e)
    step = 2.0 ** (np.floor(np.log2(largest)) - 23)
    return max(2.0 ** -11, 2.0 ** (-25 - (9 - largest * 2.0 ** -21 - 2 * step))) + 2.0 ** -10


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("order", ["ascending", "descending", "shuffled"])
@pytest.mark.parametrize("power", [10, 18, 20, 22, 23, 24])
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("codes,dtype", [("e4m3", BF), ("int8", FP)])
def test_scores(ltc, codes, dtype, call, power, order, sign):  # noqa: F811
    """Scores of 2^power times 1 .. 1.875, eight levels of them: the best
    weights are equal, and the others are 0."""
    banner(f"scores of 2^{power}, {call} {codes} {order} {sign}")
    levels = []

    def key(share):
        x = np.floor(share * 8)
        x = {"ascending": x, "descending": 7 - x, "shuffled": np.random.default_rng(power).permutation(x)}[order]
        levels.append(x)
        return 8 + x, 0 * x

    got, v, seen = attend(ltc, call, codes, dtype, power, key, sign, power)
    assert np.isfinite(got).all()
    off = rounding(1.875 * 2.0 ** power)
    for i in range(0, len(got), 5):
        x = levels[0][:seen[i]] * sign
        want = v[:seen[i]][x == x.max()].mean(0)
        assert (np.abs(got[i] - want) <= want * (off + HALF[dtype] * (1 + off))).all(), i


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [18, 20, 22, 23, 24])
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("codes,dtype", [("e4m3", BF), ("int8", FP)])
def test_near_ties(ltc, codes, dtype, call, power, sign):  # noqa: F811
    """Scores of 2^power that rise by a few nats, less than the distance at
    which the bound moves: what 32 bits make of such distances is coarse, but
    the outputs are averages of the values.  Pages' value scales differ, so bounds
    and weights are rounded apart."""
    banner(f"near ties of 2^{power}, {call} {codes} {sign}")
    got, v, seen = attend(ltc, call, codes, dtype, power, lambda share: (8 + 0 * share, np.floor(share * 5)), sign, power, 6)
    off = rounding(2.0 ** power)
    off += HALF[dtype] * (1 + off)
    assert np.isfinite(got).all()
    for i in range(0, len(got), 5):
        assert (got[i] >= v[:seen[i]].min(0) * (1 - off)).all() and (got[i] <= v[:seen[i]].max(0) * (1 + off)).all(), i
