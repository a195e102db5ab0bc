"""The dispatch's quotient x / scale: one reciprocal of the scale and one correction by the remainder give the IEEE
quotient of a bf16 x and scale = RN(amax / top), for every pair of significands, with exact rationals.

x = m 2^a and amax = n 2^b with m, n in 128..255 (bf16 values); scaling either by a power of two scales every
step by one, so one exponent of each shows them all.  top is 448 = 7 2^6 or 57344 = 7 2^13, the same
significand, so both formats have the same scales up to a power of two."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def rounded(q: Fraction) -> Fraction:
    """The nearest number of 24 significant bits, ties to even (no exponent limits)."""
    if q == 0:
        return q
    e = abs(q.numerator).bit_length() - abs(q.denominator).bit_length() - 24
    while abs(q) >= Fraction(2) ** (e + 24):
        e += 1
    while abs(q) < Fraction(2) ** (e + 23):
        e -= 1
    return Fraction(round(q / Fraction(2) ** e)) * Fraction(2) ** e  # round() ties to even


def test_rounded_is_the_float32_rounding():
    rng = np.random.default_rng(0)
    for a, b in rng.integers(1, 1 << 24, (2000, 2)):
        want = np.float32(a) / np.float32(b)  # correctly rounded
        assert rounded(Fraction(int(a), int(b))) == Fraction(float(want))


def test_corrected_quotient_is_the_ieee_quotient():
    for top in (448, 57344):
        for n in range(128, 256):
            scale = rounded(Fraction(n, top))
            r = rounded(1 / scale)
            for m in range(128, 256):
                q = rounded(m * r)
                rest = rounded(q * scale - m)       # fmaf(q, scale, -x)
                q = rounded(q - rest * r)           # fmaf(-rest, r, q)
                assert q == rounded(m / scale), (top, n, m)
