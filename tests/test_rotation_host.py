"""A rotation's rates as turns, without a GPU, against 2 pi to 50 digits that
the library has no part in."""
from fractions import Fraction

import pytest
import torch

from lossless_tensor_compression_amd import kv_cache as kc
from lossless_tensor_compression_amd import rotation as rot

TURN = Fraction("6.28318530717958647692528676655900576839433879875021")  # 2 pi, off by less than 1e-50


@pytest.mark.parametrize("rate", [1.0, 0.1, 10000.0 ** (-2 / 128), 500000.0 ** (-126 / 128), 1e-9, -1.0, -0.25, 100.0, 6.25, 1e6, 0.0,
                                  2.0 ** -80])
def test_turns_are_exact(rate):
    """A rate in turns to 2^-64 of one, and so the angle of the last position to
    2^-33 (2 pi's own digits leave 1e-43 of them)."""
    turns, = rot.turns_of([rate])
    assert 0 <= turns < 1 << 64
    off = (Fraction(turns, 1 << 64) - Fraction(rate) / TURN + Fraction(1, 2)) % 1 - Fraction(1, 2)
    assert -Fraction(1, 1 << 64) - Fraction(1, 10 ** 40) <= off <= Fraction(1, 10 ** 40)
    position = 2 ** 31 - 2
    angle = Fraction(position * turns % (1 << 64), 1 << 64)
    off = (angle - position * Fraction(rate) / TURN + Fraction(1, 2)) % 1 - Fraction(1, 2)
    assert abs(off) <= Fraction(1, 1 << 33) + Fraction(1, 10 ** 30)


def test_large_rates():
    """The largest there is: its turns are what its 1,024 bits say (by pi to more digits, from the formula of
    Euler: 20 arctan(1/7) + 8 arctan(3/79))."""
    def arctan(x, terms):
        return sum(Fraction((-1) ** k, 2 * k + 1) * x ** (2 * k + 1) for k in range(terms))

    rate = 1.7e308
    pi = 20 * arctan(Fraction(1, 7), 250) + 8 * arctan(Fraction(3, 79), 160)  # off by 7^-500, 2^-1403
    want = Fraction(rate) / (2 * pi)
    turns, = rot.turns_of([rate])
    off = (Fraction(turns, 1 << 64) - want + Fraction(1, 2)) % 1 - Fraction(1, 2)
    assert abs(off) <= Fraction(1, 1 << 63)


def test_a_rotation_that_is_on_no_gpu(monkeypatch):
    """Refused, where a search for its GPU would not end."""
    monkeypatch.setattr(kc, "_current_gpu", lambda: 0)
    r = rot.Rotation(64, device="cpu")
    q, lengths = torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.tensor([3, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        rot.norm_rotate(q, q, r, lengths)
