"""The division of the block quantiser (csrc/quantize.hip) on the CPU: three operations an element round x / d to nearest,
for every pair of an element and a block maximum.

x is bf16, d = fl(max / 448) with max bf16.  In the range where the kernel divides so, nothing underflows, and powers of
two only move exponents: 128 mantissas of max times 128 of x, on both sides of a power of two, are all there is.  Floats
are computed as integers and exact fractions here.
"""
from fractions import Fraction

import pytest


def rn(v, bits=24):
    """The positive fraction v rounded to nearest, ties to even, at `bits` bits (no range limits)."""
    e = v.numerator.bit_length() - v.denominator.bit_length()
    if Fraction(2) ** e > v:
        e -= 1  # 2^e <= v < 2^(e + 1)
    unit = Fraction(2) ** (e - bits + 1)
    n, r = divmod(v, unit)
    if r * 2 > unit or (r * 2 == unit and n % 2):
        n += 1
    return n * unit, unit


def signed_rn(v):
    return Fraction(0) if v == 0 else (rn(v)[0] if v > 0 else -rn(-v)[0])


@pytest.mark.parametrize("half", range(4))
def test_three_operations_round_the_quotient(half):
    worst, inexact = Fraction(0), 0
    for m in range(128 + 32 * half, 128 + 32 * half + 32):
        d = rn(Fraction(m, 448))[0]
        r = rn(1 / d)[0]
        for x in range(128, 256):
            quotient, unit = rn(x / d)
            t = rn(x * r)[0]
            worst = max(worst, abs(t - x / d) / unit)
            left = signed_rn(x - t * d)  # (exact in all but a few pairs)
            inexact += left != x - t * d
            assert rn(t + r * left)[0] == quotient, (m, x)
    assert worst < Fraction(3, 2)
    print(f"t is off by up to {float(worst):.3f} units, {inexact} remainders were rounded")
