"""The rotation's frequencies as fractions of 2^64 of a turn against whole-number
arithmetic of 1400 bits, and what is left of it at the farthest positions."""
import math
import random
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def grs():
    from gradient_reduction_sharded_gb300 import _build
    _build.build()
    from gradient_reduction_sharded_gb300 import grs as g
    return g


BITS = 1400


def arctan_of_one_over(n):
    """arctan(1 / n) in units of 2^-BITS, by its series."""
    term = total = (1 << BITS) // n
    k = 1
    while term:
        term //= -n * n
        k += 2
        total += term // k
    return total


PI = Fraction(4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)), 1 << BITS)  # Machin


def off(turns, freq, position=1):
    """Distance, in turns, of position * turns / 2^64 from position * freq / (2 pi)."""
    d = (Fraction(position * turns, 1 << 64) - position * Fraction(freq) / (2 * PI)) % 1
    return min(d, 1 - d)


def test_turns_to_two_to_the_minus_64(grs):
    rng = random.Random(7)
    freqs = [1.0, 0.0, -0.0, -1.0, 2 * math.pi, -2 * math.pi, math.nextafter(2 * math.pi, 0), 1e-300, -1e-300, 5e-324, 6.5, 1e9, -1e15, 2.0 ** 60, -1e-30]
    freqs += [base ** (-2 * i / 128) for base in (1e4, 5e5, 1e6) for i in range(64)]
    freqs += [10 ** rng.uniform(-12, 6) * rng.choice((-1, 1)) for _ in range(300)]
    for f, t in zip(freqs, grs.grs_rope_turns(freqs)):
        # Two roundings to 2^-64; 1 / (2 pi) in two doubles and their product: 2^-107 of the frequency.
        limit = Fraction(1, 1 << 64) + Fraction(abs(f)) / 2 ** 107
        assert off(t, f) <= limit, (f, float(off(t, f) / limit))
        for position in (-2 ** 31, 2 ** 31 - 1, 123456789):
            assert off(t, f, position) <= abs(position) * limit


def test_turns_of_opposite_frequencies_are_opposite(grs):
    freqs = [0.3, 1.0, 1e-7, 6.0, 700.25]
    a, b = grs.grs_rope_turns(freqs), grs.grs_rope_turns([-f for f in freqs])
    assert all((x + y) % 2 ** 64 == 0 for x, y in zip(a, b))
