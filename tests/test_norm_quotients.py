"""The step by which the norm forms E4M3 codes of quotients (q = RN(x RN(1/a)), then RN(q + RN(x - q a) RN(1/a))), in whole
numbers: wherever it could miss the nearest fp32 number next to a border between two codes, it does not."""
from fractions import Fraction


def nearest(x):
    """x (positive or negative) rounded to 24 bits, nearest even."""
    if x == 0:
        return Fraction(0)
    sign, x = (1, x) if x > 0 else (-1, -x)
    e = x.numerator.bit_length() - x.denominator.bit_length() - 24
    while x >= Fraction(2) ** (e + 24):
        e += 1
    while x < Fraction(2) ** (e + 23):
        e -= 1
    return sign * round(x / Fraction(2) ** e) * Fraction(2) ** e      # (round: to even)


def step(x, a):
    inv = nearest(1 / a)
    q = nearest(x * inv)
    return nearest(q + nearest(x - q * a) * inv)


def test_quotients_next_to_the_middle_beside_a_border():
    """A border between two codes is b 2^k with b of five bits (16 .. 31, fewer among the subnormals). In units of 2^-20 of a
    border, the middle between it and its neighbour times a (24 bits, A) is P = b A 2^20 +- A. The step's result is that of
    a quotient off by 3 * 2^-24 of a unit at most, that is by 12 in P, and x is a multiple of 2^24 (2^25 from 2^48 on). P
    comes that close to one only if A is within 12 of a multiple of 2^20. (The middle below b = 16, in the smaller binade,
    is A (2^25 - 1) in half units, and A itself its distance from the next x.)"""
    seen = 0
    for m in range(8, 17):
        for d in range(-24, 25):
            A = (m << 20) + d
            if not 1 << 23 <= A < 1 << 24:
                continue
            for b in range(16, 32):
                for side in (1, -1):
                    P = b * A * 2 ** 20 + side * A
                    unit = 2 ** 24 if P < 2 ** 48 else 2 ** 25
                    x = (P + unit // 2) // unit * unit
                    if abs(P - x) > 24:
                        continue
                    seen += 1
                    x, a = Fraction(x), Fraction(A)
                    assert step(x, a) == nearest(x / a), (A, b, side)
    assert seen > 100


def test_quotients_on_and_next_to_a_border():
    import random
    rng = random.Random(1)
    for _ in range(3000):
        A, b = rng.randrange(1 << 23, 1 << 24), rng.randrange(16, 32)
        x = nearest(Fraction(b * A))
        for _ in range(rng.randrange(3)):
            x = nearest(x * (1 + Fraction(rng.choice((-1, 1)), 1 << 23)))
        assert step(x, Fraction(A)) == nearest(x / A)
    for b in range(16, 32):     # exactly on it
        for A in (1 << 23, (1 << 24) - 1, 0xABCDE0, 0x800020):
            if nearest(Fraction(b * A)) == b * A:
                assert step(Fraction(b * A), Fraction(A)) == b
