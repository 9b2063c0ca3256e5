"""The 8-bit quantization's rounding, on the CPU: q = rint(127 v / top) of bf16
v and top, by the kernel's arithmetic (fp32, step by step, in exact rationals),
for every pair of significands and every exponent difference at which q is not
plainly zero.  Powers of two beyond that only shift the exponents."""
from fractions import Fraction

import numpy as np


def _f32(v: Fraction) -> Fraction:
    """v rounded to 24 significant bits, ties to even (no value here is subnormal or overflows)."""
    if v == 0:
        return v
    n, d = abs(v.numerator), v.denominator
    e = n.bit_length() - d.bit_length()
    if Fraction(n, d) < Fraction(2) ** e:
        e -= 1
    ulp = Fraction(2) ** (e - 23)
    return (round(abs(v) / ulp) * ulp) * (1 if v > 0 else -1)   # round() of a Fraction: to even


def test_rounding_is_the_exact_quotients():
    least = Fraction(1)
    for b in range(128, 256):
        inv = _f32(Fraction(1, b))
        for d in range(0, 10):
            for a in range(128, 256):
                if d == 0 and a > b:
                    continue
                top = Fraction(b * 2 ** d)
                exact = 127 * a / top
                t = Fraction(127 * a)                      # 15 bits: exact
                q0 = _f32(t * inv / 2 ** d)
                q = _f32(_f32(t - q0 * top) * inv / 2 ** d + q0)
                assert round(_f32(q + 12582912) - 12582912) == round(exact), (a, b, d)
                tie = abs(exact - (exact.__floor__() + Fraction(1, 2)))
                if tie and exact >= Fraction(1, 4):
                    least = min(least, tie / exact)
                assert abs(q - exact) <= exact * Fraction(1, 2 ** 23)
    # the argument's bound, which the corrected quotient's error stays far within
    assert least >= Fraction(1, 254 * 255) > Fraction(1, 2 ** 16)


def test_a_quotient_close_to_a_tie():
    """161/64 against 213: 7.3e-5 from 1.5, and still rounded down."""
    v, top = np.float32(161 / 64), np.float32(213)
    inv = np.float32(1) / top
    t = v * np.float32(127)
    q0 = t * inv
    q = np.float32(np.float64(np.float32(np.float64(t) - np.float64(q0) * np.float64(top))) * np.float64(inv) + np.float64(q0))
    assert 0 < 1.5 - 127 * float(v) / float(top) < 1e-4
    assert float(np.float32(q + np.float32(12582912.0))) - 12582912.0 == 1.0
