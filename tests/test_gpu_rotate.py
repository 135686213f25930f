"""Norm and rotation of queries and keys on the GPU against 64 bits.

Tolerances, of the sum |a| + |b| of the numbers turned together: the phase is
rounded to 2^-24 of half a turn at most (2^-22.3), sine and cosine are off by 4
ulp (2^-22), the norm's sum by 14 roundings of 2^-24, the root, the quotient and
the four products by 8 more: below 2^-19 in all; then half a step of the type."""
import math

import numpy as np
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}
SMALLEST = {BF: 2.0 ** -133, FP: 2.0 ** -24}


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def angles(position, rates):
    """position * rate modulo a turn: the rate's turns are exact to 2^-53 of themselves, the product is of whole numbers."""
    out = []
    for r in rates:
        n, d = float(r / (2 * math.pi)).as_integer_ratio()
        out.append(2 * math.pi * (n * int(position) % d / d))
    return np.array(out)


def oracle(x, positions, rates, rotary, pairs, weight, eps):
    """(y, sum of magnitudes turned together)."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight
    out, size = y.copy(), np.abs(y)
    i = np.arange(rotary // 2)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rotary // 2)
    for r, p in enumerate(positions):
        if p is None:
            out[r] = size[r] = 0
            continue
        th = angles(p, rates)
        out[r][:, a] = y[r][:, a] * np.cos(th) - y[r][:, b] * np.sin(th)
        out[r][:, b] = y[r][:, b] * np.cos(th) + y[r][:, a] * np.sin(th)
        size[r][:, a] = size[r][:, b] = np.abs(y[r][:, a]) + np.abs(y[r][:, b])
    return out, size


def check(ltc, dtype, dim, q_heads, heads, new, past, rotary=None, pairs=False, norm=(True, True), theta=10000.0, size=1.0,
          eps=1e-6, single=False, seed=0, front=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    rotary = dim if rotary is None else rotary
    rows = sum(new) + front + behind
    rot = ltc.Rotation(dim, theta=theta, rotary=rotary, pairs=pairs)
    q, k = ((size * torch.randn(rows, h, dim, generator=g)).to(dtype).cuda() for h in (q_heads, heads))
    qw, kw = ((1 + 0.3 * torch.randn(dim, generator=g)).to(dtype).cuda() if n else None for n in norm)
    lengths = torch.tensor([a + b for a, b in zip(new, past)], dtype=torch.int32, device="cuda")
    cu = None if single else torch.cumsum(torch.tensor([0] + new), 0).add(front).to(torch.int32).cuda()
    got = ltc.norm_rotate(q, k, rot, lengths, cu, q_weight=qw, k_weight=kw, eps=eps)
    positions = [None] * front + [p + t for n, p in zip(new, past) for t in range(n)] + [None] * behind
    rates = [theta ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    for x, y, w in zip((q, k), got, (qw, kw)):
        want, mag = oracle(x.double().cpu().numpy(), positions, rates, rotary, pairs,
                           None if w is None else w.double().cpu().numpy(), eps)
        off = np.abs(y.double().cpu().numpy() - want)
        limit = 2.0 ** -19 * mag + HALF[dtype] * (np.abs(want) + 2.0 ** -19 * mag) + SMALLEST[dtype]
        assert (off <= limit).all(), (np.argwhere(off > limit)[:5], off[off > limit][:5], limit[off > limit][:5])
    rot.check()
    return q, k, got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (96, 96), (128, 128), (192, 192), (256, 256), (128, 64), (96, 48), (192, 16),
                                        (256, 240), (64, 0)])
def test_dims(ltc, dim, rotary, pairs, dtype):
    banner(f"rotate {rotary} of {dim}, pairs {pairs}")
    check(ltc, dtype, dim, 6, 2, [3, 1, 20], [0, 5, 100], rotary, pairs)


@pytest.mark.parametrize("q_heads,heads", [(1, 1), (32, 8), (7, 7), (64, 1), (33, 3)])
@pytest.mark.parametrize("dim", [96, 128])
def test_heads(ltc, q_heads, heads, dim):
    check(ltc, BF, dim, q_heads, heads, [1, 5], [3, 0])


@pytest.mark.parametrize("position", [0, 1, 131071, 2 ** 20 + 1, 2 ** 30, 2 ** 31 - 2])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5])
def test_far_positions(ltc, position, theta):
    check(ltc, FP, 128, 2, 1, [1, 1], [position, max(position - 1, 0)], theta=theta, single=True)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_without_norm(ltc, norm):
    check(ltc, BF, 128, 4, 2, [9], [70], norm=norm)


@pytest.mark.parametrize("dtype,size", [(BF, 1e-30), (BF, 1e15), (FP, 1e-4), (FP, 1e3), (BF, 0.0)])
def test_sizes(ltc, dtype, size):
    """Rows of zeros, and rows whose squares are far from one (eps 0: the quotient alone)."""
    if size in (1e-30, 1e-4):
        check(ltc, dtype, 64, 2, 2, [5], [7], size=size)
        return
    check(ltc, dtype, 64, 2, 2, [5], [7], size=size, eps=0.0 if size else 1e-6)


def test_many_sequences(ltc):
    """Sequences without rows, more sequences than rows, rows of no sequence."""
    check(ltc, BF, 64, 2, 1, [(i * 7) % 4 for i in range(200)], [(i * 31) % 5000 for i in range(200)])
    check(ltc, BF, 64, 2, 1, [0] * 100 + [2] + [0] * 50, [i for i in range(151)])
    check(ltc, FP, 96, 2, 1, [2, 0, 3], [5, 6, 7], front=3, behind=4)


@pytest.mark.parametrize("dim", [64, 96, 192])
def test_many_rows(ltc, dim):
    """More than the rows that four waves share."""
    check(ltc, BF, dim, 5, 2, [700, 1, 0, 400], [5, 60000, 3, 0], pairs=dim == 96)


def test_strided_parts_of_one_tensor(ltc):
    qkv = torch.randn(10, 12, 128, device="cuda").to(BF)
    rot = ltc.Rotation(128)
    lengths = torch.full((10,), 50, dtype=torch.int32, device="cuda")
    a = ltc.norm_rotate(qkv[:, :8], qkv[:, 8:10], rot, lengths)
    b = ltc.norm_rotate(qkv[:, :8].contiguous(), qkv[:, 8:10].contiguous(), rot, lengths)
    odd = torch.empty(10 * 8 * 128 + 1, dtype=BF, device="cuda")[1:].view(10, 8, 128).copy_(qkv[:, :8])
    c = ltc.norm_rotate(odd, qkv[:, 8:10], rot, lengths)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_nan_and_infinity_stay_in_their_head(ltc):
    rot, w = ltc.Rotation(64), torch.ones(64, dtype=BF, device="cuda")
    q, k = torch.randn(3, 4, 64, device="cuda").to(BF), torch.randn(3, 2, 64, device="cuda").to(BF)
    q[1, 2, 5], k[0, 1, 9] = float("nan"), float("inf")
    lengths = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    a, b = ltc.norm_rotate(q, k, rot, lengths, q_weight=w, k_weight=w)
    nan = torch.isnan(a).any(-1)
    assert nan.sum() == 1 and bool(nan[1, 2]) and torch.isnan(a[1, 2]).all()
    nan = torch.isnan(b).any(-1)
    assert nan.sum() == 1 and bool(nan[0, 1])


def test_bad_sequences_are_reported_and_zero(ltc):
    rot = ltc.Rotation(64)
    q = torch.randn(10, 2, 64, device="cuda").to(BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    for lengths, cu, zero in (([5, 1, 9], [0, 3, 6, 10], range(3, 6)), ([5, -1, 9], [0, 3, 6, 10], range(3, 6)),
                              ([5, 5, 9], [0, 3, 6, 11], range(6, 10))):
        a, b = ltc.norm_rotate(q, q, rot, torch.tensor(lengths, **i32), torch.tensor(cu, **i32))
        for x in (a, b):
            assert [not bool(x[r].any()) for r in range(10)] == [r in zero for r in range(10)]
        with pytest.raises(ltc.LTCError):
            rot.check()
        rot.check()
    ltc.norm_rotate(q, q, rot, torch.tensor([5] * 12, **i32), torch.tensor([0] * 11 + [12, 10], **i32))  # more sequences than rows
    with pytest.raises(ltc.LTCError):
        rot.check()


def test_given_rates(ltc):
    """Rates of a stretched context, and negative ones."""
    rates = [0.25 * 10000.0 ** (-i / 32) for i in range(31)] + [-1.0]
    rot = ltc.Rotation(64, rates=rates)
    q = torch.randn(3, 1, 64, device="cuda").to(FP)
    lengths = torch.tensor([900001, 1, 77], dtype=torch.int32, device="cuda")
    a, _ = ltc.norm_rotate(q, q, rot, lengths)
    want, mag = oracle(q.double().cpu().numpy(), [900000, 0, 76], rates, 64, False, None, 0)
    assert (np.abs(a.double().cpu().numpy() - want) <= 2.0 ** -18 * mag + HALF[FP] * np.abs(want) + SMALLEST[FP]).all()


def test_captured(ltc):
    rot, w = ltc.Rotation(128), torch.ones(128, dtype=BF, device="cuda")
    q, k = torch.randn(5, 8, 128, device="cuda").to(BF), torch.randn(5, 2, 128, device="cuda").to(BF)
    lengths = torch.tensor([5, 60, 7, 1000, 1], dtype=torch.int32, device="cuda")
    ltc.norm_rotate(q, k, rot, lengths, None, w, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = ltc.norm_rotate(q, k, rot, lengths, None, w, w)
    for _ in range(4):
        lengths.add_(1)
        q.copy_(torch.randn_like(q))
        graph.replay()
        x, y = ltc.norm_rotate(q, k, rot, lengths, None, w, w)
        assert torch.equal(a, x) and torch.equal(b, y)
        torch.cuda.synchronize()


def test_refusals(ltc):
    rot = ltc.Rotation(64)
    q = torch.randn(2, 2, 64, device="cuda").to(BF)
    lengths = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    for args, kw in (((q.half(), q), {}), ((q.cpu(), q), {}), ((q[:1], q), {}), ((q[..., :32], q), {}), ((q, q[0]), {}),
                     ((q, q), dict(q_weight=w.float())), ((q, q), dict(k_weight=w[:32])), ((q.clone().requires_grad_(), q), {}),
                     ((q, q), dict(q_weight=w.clone().requires_grad_()))):
        with pytest.raises(ValueError):
            ltc.norm_rotate(*args, rot, lengths, **kw)
    for n, cu in ((lengths[:1], None), (lengths.long(), None), (lengths, lengths)):
        with pytest.raises(ValueError):
            ltc.norm_rotate(q, q, rot, n, cu)
    with pytest.raises(ltc.LTCError):
        ltc.norm_rotate(q.float(), q.float(), rot, lengths)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ltc.LTCError):
            ltc.norm_rotate(q, q, rot, lengths, eps=eps)
    a, b = ltc.norm_rotate(q[:0], q[:0], rot, lengths[:0])
    assert a.shape == (0, 2, 64) and b.shape == (0, 2, 64)
