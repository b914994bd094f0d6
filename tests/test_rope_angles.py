"""The bound on a rotary angle that the header states, by exact arithmetic (CPU): the
frequency as a 64-bit fraction of a turn, its product with the position modulo 2^64,
the upper 32 bits as fp32 half turns."""
from fractions import Fraction

import numpy as np
import pytest

import rope_reference as ref


def kernel_turns(position, freq):
    """The angle that the kernel hands to its sine and cosine, in turns (the frequency's last bit or two aside)."""
    f = Fraction(float(np.float32(freq)))
    whole = (abs(f.numerator) * ref._INV // f.denominator) >> (ref._BITS - 64)
    fraction = (whole if f > 0 else -whole) * position % (1 << 64)
    upper = fraction >> 32
    upper -= (upper >> 31) << 32
    return float(np.float32(upper)) * 2.0 ** -32


@pytest.mark.parametrize("freq", [1.0, 0.7, 1e-4, 3e-6, -0.33, 1000.1, 1e6])
def test_within_its_bound(freq):
    rng = np.random.default_rng(int(abs(freq) * 1e6))
    positions = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, *map(int, rng.integers(-2 ** 31, 2 ** 31, 3000))]
    worst = 0.0
    for pos in positions:
        diff = abs(kernel_turns(pos, freq) - ref.turn_fraction(pos, freq))
        worst = max(worst, min(diff, 1.0 - diff))
    assert worst <= 2.0 ** -26 + 2.0 ** -31     # fp32 half turns; the rest
    assert worst > 2.0 ** -28                   # (the rounding to fp32 is what it comes from)
