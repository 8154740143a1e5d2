"""The few-token layer's FP8 quotients: x / s as q + r (x - q s), q = RN(x r), r = RN(1 / s), all in fp32 with fused
multiply-adds, give the codes of IEEE division for every x and s.

q is off by at most 1.5 units in its last place (ulp): half a one from r, scaled by up to 2, and half a one of its own.  The
remainder x - q s has at most 25 bits, so with its own rounding and r's the correction is right to 3 2^-24 of itself, and
the corrected quotient, before its last rounding, to 1.5 * 3 2^-24 < 2^-21 ulp.  It can then differ from RN(x / s) only where
x / s lies nearer than that to the middle of two floats, and a code only where, besides, the nearer or farther of the two is
a tie between neighbouring codes: their mantissas are 1 + j / 16.  The mantissas of s and x near those 34 middles are few;
all of them are tried here, in exact arithmetic."""
from fractions import Fraction

import numpy as np


def _rn(v):
    """A positive fraction rounded to 24 bits, ties to even."""
    if v == 0:
        return v
    e = v.numerator.bit_length() - v.denominator.bit_length()
    unit = Fraction(2) ** (e - 23 if v >= Fraction(2) ** e else e - 24)
    return round(v / unit) * unit          # (Fraction rounds ties to even)


def _signed(v):
    return -_rn(-v) if v < 0 else _rn(v)


def _divide(x, s):
    r = _rn(1 / s)
    q = _rn(x * r)
    return _signed(_signed(x - q * s) * r + q)


def _hard_cases():
    """(X, S, middle) as integers of 24 bits with X / S (times a power of two) within 2^-21 ulp of a middle beside a tie."""
    s = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    for j in range(16):
        tie = (16 + j) << 21                                     # 1 + j / 16 in units of 2^-25: an ulp is 4, below 1 it is 2
        for mid in (tie + 2, tie - 2 if j else tie - 1):
            p = mid * s                                          # x would be p 2^-25 (2^-26: a binade up)
            for shift in (25, 26):
                low = p & ((1 << shift) - 1)
                off = np.minimum(low, (1 << shift) - low)        # |x / s - middle| = off / s in units of 2^-25
                for i in np.flatnonzero(off * (1 << 19) <= s):   # 2^-21 ulp
                    x = int((int(p[i]) + (1 << (shift - 1))) >> shift)
                    if 1 << 23 <= x < 1 << 24:
                        yield x, int(s[i])


def test_every_quotient_near_a_border_of_two_codes():
    n = 0
    for x, s in _hard_cases():
        assert _divide(Fraction(x), Fraction(s)) == _rn(Fraction(x, s)), (x, s)
        n += 1
    assert n > 20


def test_quotients_of_all_kinds():
    """Random mantissas, and the ends of their range."""
    g = np.random.default_rng(1)
    x, s = (g.integers(1 << 23, 1 << 24, 4000).tolist() for _ in range(2))
    ends = [1 << 23, (1 << 23) + 1, (1 << 24) - 2, (1 << 24) - 1]
    pairs = list(zip(x, s)) + [(a, b) for a in ends for b in ends] + list(zip(ends * 500, s)) + list(zip(x, ends * 500))
    for a, b in pairs:
        assert _divide(Fraction(a), Fraction(b)) == _rn(Fraction(a, b)), (a, b)
