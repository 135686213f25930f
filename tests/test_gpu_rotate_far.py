"""Angles of far positions on the GPU, against 2 pi to 50 digits.

Tolerance, of |a| + |b| of the numbers turned together: an angle is rounded to
2^-26 of a turn (2^-23.3) and its product to 2^-32 of one, sine and cosine are off
by 4 ulp (2^-22), two products and a sum by 3 roundings of 2^-24: below 2^-20 in
all; then half a step of the type."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from gpu_util import banner
from test_rotation_host import TURN

pytestmark = pytest.mark.gpu

HALF, SMALLEST = 2.0 ** -11, 2.0 ** -24


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("position", [0, 1, 131071, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 2])
def test_angles(ltc, position, pairs):
    banner(f"rotate position {position}, pairs {pairs}")
    rates = [1.0, 0.1, 6.25, -1.0, 100.0, 1e-3, 2.0 ** -40, 0.0] * 8
    x = torch.randn((1, 3, 128), generator=torch.Generator().manual_seed(position % 1000)).to(torch.float16).cuda()
    rot = ltc.Rotation(128, rates=rates, pairs=pairs)
    lengths = torch.tensor([position + 1], dtype=torch.int32, device="cuda")
    y, _ = ltc.norm_rotate(x, x, rot, lengths)
    angle = np.array([float(position * Fraction(r) / TURN % 1) for r in rates]) * 2 * math.pi
    i = np.arange(64)
    ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + 64)
    x = x.double().cpu().numpy()[0]
    a, b = x[:, ia], x[:, ib]
    want, size = np.zeros((3, 128)), np.zeros((3, 128))
    want[:, ia], want[:, ib] = a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)
    size[:, ia] = size[:, ib] = np.abs(a) + np.abs(b)
    off = np.abs(y.double().cpu().numpy()[0] - want)
    assert (off <= 2.0 ** -20 * size + HALF * (np.abs(want) + 2.0 ** -20 * size) + SMALLEST).all()
    rot.check()


@pytest.mark.parametrize("dim", [128, 256])
def test_many_rows(ltc, dim):
    """The main sizes in calls of more rows than four waves share: the same bits as a call of a few of them."""
    rot, g = ltc.Rotation(dim), torch.Generator(device="cuda").manual_seed(5)
    rows = [700, 1, 0, 400]
    q, k = (torch.randn((sum(rows), h, dim), generator=g, device="cuda").to(torch.bfloat16) for h in (5, 2))
    w = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16)
    lengths = torch.tensor([705, 60001, 3, 400], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 700, 701, 701, 1101], dtype=torch.int32, device="cuda")
    many = ltc.norm_rotate(q, k, rot, lengths, cu, w, w)
    for i, (lo, hi) in enumerate(((0, 700), (700, 701), (701, 701), (701, 1101))):
        if hi > lo:
            few = ltc.norm_rotate(q[lo:hi], k[lo:hi], rot, lengths[i:i + 1], torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"), w, w)
            assert all(torch.equal(x[lo:hi], y) for x, y in zip(many, few))
    rot.check()
