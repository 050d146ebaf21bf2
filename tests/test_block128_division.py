"""The FP8 block-128 quantizers' two quotients of a block's magnitude A, s = fl32(A / 448) and r = fl32(448 / A),
as the kernel forms them (one fused-multiply-add correction of a reciprocal product), against correctly
rounded division in exact rational arithmetic, for every bf16 A from the floor 2^-100 up."""
from fractions import Fraction

import numpy as np


def round32(x: Fraction) -> Fraction:
    """Nearest fp32 (ties to even) of a non-negative or negative rational in the normal range."""
    if x == 0:
        return x
    sign, x = (-1, -x) if x < 0 else (1, x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    ulp = Fraction(2) ** (max(e, -126) - 23)
    q, rem = divmod(x, ulp)
    if 2 * rem > ulp or (2 * rem == ulp and q % 2 == 1):
        q += 1
    return sign * q * ulp


def magnitudes():
    bits = np.arange(27 << 7, 255 << 7, dtype=np.uint32)  # 2^-100 = exponent field 27, to the largest finite
    return (bits << 16).view(np.float32)


def test_scale_quotient():
    inv = round32(Fraction(1, 448))
    for a in magnitudes():
        a = Fraction(float(a))
        q = round32(a * inv)
        e = round32(a - 448 * q)
        assert round32(q + e * inv) == round32(a / 448)


def test_reciprocal_quotient_for_reciprocals_two_ulps_off():
    # every significand at one exponent: scaling A by a power of two scales every step exactly (the normal range
    # is never left: A 2^-14 lies in [2^-114, 2^114), its reciprocal too, the quotient in [2^-120, 2^109))
    c = Fraction(448, 1 << 14)
    for exponent in (27, 127, 254):
        for m in range(128):
            a = Fraction(128 + m, 128) * Fraction(2) ** (exponent - 127)
            d = a / (1 << 14)
            best = round32(1 / d)
            e = best.numerator.bit_length() - best.denominator.bit_length()
            ulp = Fraction(2) ** (e - 24)
            for off in range(-4, 5):  # in half ulps' neighbourhood: ulp may be half the spacing
                t = round32(best + off * ulp)
                u = round32(c * t)
                r = round32(u + round32(c - d * u) * t)
                assert r == round32(Fraction(448) / a), (float(a), off)
