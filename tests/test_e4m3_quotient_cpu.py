"""The 8-bit norm's quotient (a product with the rounded reciprocal and one
correction) rounds to e4m3 as the rounded quotient does: every pair of
mantissas for which it could do otherwise, in exact arithmetic.

Before its rounding the corrected product is within 2^-22 ulp of the quotient
(q is off by at most 1.5 ulp; of that the residual's rounding and the
reciprocal's leave 2^-24 each), so the binary32 results differ at most where
the quotient lies that close to the middle of two neighbours, and the e4m3
results only if one neighbour is halfway between two e4m3 values: an odd
number of at most five bits."""
from fractions import Fraction

import numpy as np


def rounded(x):
    """x to the nearest binary32, ties to even (no limits of the exponent)."""
    sign, x, e = (-1 if x < 0 else 1), abs(x), 0
    if x == 0:
        return x
    while x >= 2:
        x, e = x / 2, e + 1
    while x < 1:
        x, e = x * 2, e - 1
    i = int(x * 2 ** 23)
    rest = x * 2 ** 23 - i
    i += rest > Fraction(1, 2) or (rest == Fraction(1, 2) and i % 2)
    return sign * Fraction(i, 2 ** 23) * Fraction(2) ** e


def test_the_corrected_product_is_the_quotient_next_to_e4m3_ties():
    b = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    cases = 0
    for tie in range(16, 32):                    # a tie's mantissa, in sixteenths
        for side in (1, -1):
            # the middle beside it, in units of 2^-25 (below 1 the steps halve)
            middle = tie * (1 << 21) + (-1 if tie == 16 and side < 0 else 2 * side)
            for less in (0, 1):                  # a < b: the quotient is a / b * 2
                product = b * middle
                a = (product + (1 << (24 + less))) >> (25 + less)
                off = np.abs((a << (25 + less)) - product)
                near = (a >= 1 << 23) & (a < 1 << 24) & (off <= (b >> 19))     # 2^-21 ulp
                for u, d in zip(a[near].tolist(), b[near].tolist()):
                    u, d = Fraction(u, 2 ** 23), Fraction(d, 2 ** 23)
                    inv = rounded(1 / d)
                    q = rounded(u * inv)
                    assert rounded(q - rounded(q * d - u) * inv) == rounded(u / d), (u, d)
                    cases += 1
    assert cases > 100
