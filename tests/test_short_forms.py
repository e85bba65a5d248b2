"""The 8-bit update's short root and quotient (no GPU): an exact model of the
quotient's roundings, in integers, against the bound that says which quotients
could be misrounded at all.

Notation: mantissas A, D in [2^23, 2^24); y = the correctly rounded 1/d;
q0 = rn(a y), r = rn(a - q0 d), q1 = rn(q0 + r y) (Newton's reciprocal and
Markstein's correction by the residual).  Lengths are in last-place units of the
quotient, and the quotient lies an integer number of 1/(2D) from the nearest
middle between two floats.

- a y is off by at most 1 unit from y's rounding (a 2^-25 < 2^-24) and half a
  unit from its own: 1.5 units.
- The residual is therefore an integer of up to 1.5 * 2^24 (in units of the last
  places of q and d): above 2^24 an odd one is rounded, by 1.
- Before the last rounding the error is r (y - 1/d) <= 1.5 * 2/(2D) plus that of
  the residual, times y: 2/(2D) (1 + 2^-24).  In all below 5.01/(2D)."""
import random
from fractions import Fraction

import pytest

P = 24


def rn(x: Fraction) -> Fraction:
    """x > 0 (or 0, or negative) rounded to 24 bits, ties to even."""
    if x == 0:
        return x
    if x < 0:
        return -rn(-x)
    n, d = x.numerator, x.denominator
    e = n.bit_length() - d.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    ulp = Fraction(2) ** (e - P + 1)
    k = x / ulp
    f = k.numerator // k.denominator
    half = k - f - Fraction(1, 2)
    return ulp * (f + (1 if half > 0 or (half == 0 and f & 1) else 0))


def quotient(A, D):
    """(units between the exact quotient and the value before the last rounding,
    the residual in units, the short form, the correctly rounded quotient)."""
    a, d = Fraction(A), Fraction(D)
    y = rn(1 / d)
    q0 = rn(a * y)
    exact_r = a - q0 * d
    r = rn(exact_r)
    z = q0 + r * y
    unit = Fraction(1, 2 ** 23) if A >= D else Fraction(1, 2 ** 24)
    return abs(z - a / d) / unit, exact_r / unit, rn(z), rn(a / d)


def hard_pairs(rng, count):
    """Pairs whose quotient lies 1/(2D) to 8/(2D) from a middle: 2^(s+1) A =
    (2K+1) D + delta, s = 23 for A >= D and 24 below it, solved for A modulo D."""
    while count:
        D = rng.randrange(1 << 23, 1 << 24) | 1
        delta = rng.choice([k for k in range(-8, 9) if k])
        s = rng.choice([23, 24])
        # (2K+1) D + delta = 0 mod 2 needs D + delta even; then A = ((D + delta)/2) 2^-s mod D
        if (D + delta) & 1:
            continue
        A = (D + delta) // 2 * pow(2, -s, D) % D
        while A < 1 << 23:
            A += D
        if A < 1 << 24 and (A >= D) == (s == 23):
            yield A, D
            count -= 1


def check(A, D):
    off, r, got, want = quotient(A, D)
    assert off * 2 * D < Fraction(501, 100), (A, D)
    assert r.denominator == 1 and abs(r) <= 3 << 23, (A, D)
    assert got == want, (A, D)
    return abs(r)


def test_the_residual_may_be_rounded_and_the_quotient_is_not():
    """One residual that does not fit into 24 bits."""
    assert check(12693471, 14795003) == 17800639


@pytest.mark.parametrize("seed", range(3))
def test_any_pairs(seed):
    rng = random.Random(seed)
    rounded = sum(check(rng.randrange(1 << 23, 1 << 24), rng.randrange(1 << 23, 1 << 24)) > 1 << 24 for _ in range(8000))
    assert rounded


def test_pairs_next_to_a_middle():
    for A, D in hard_pairs(random.Random(7), 6000):
        check(A, D)


def test_edges():
    top = (1 << 24) - 1
    for A in (1 << 23, (1 << 23) + 1, 3 << 22, top - 1, top):
        for D in (1 << 23, (1 << 23) + 1, 3 << 22, top - 1, top):
            check(A, D)
