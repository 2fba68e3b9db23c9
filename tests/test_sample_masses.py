"""How far the draw's masses, sums of weights rounded to multiples of 2^-44, are from those in real numbers: the bound that
the header states, on rows with long flat tails of light tokens, where the roundings all have one sign."""
import random
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

from tests.sample_masses import ONE, Row, build

getcontext().prec = 40


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return build(tmp_path_factory.mktemp("masses"))


def real_masses(x, order, t):
    """Cumulated masses of the tokens in order, in units of 2^-44 of the first one's weight (exact to 35 digits)."""
    v = x[order]
    w = {float(a): Decimal(2) ** 44 * ((Decimal(float(a)) - Decimal(float(v[0]))) / Decimal(float(np.float32(t)))).exp() for a in np.unique(v)}
    out, sum_ = [], Decimal(0)
    for a in v:
        sum_ += w[float(a)]
        out.append(sum_)
    return out


def borders(lib, x, t):
    """(the largest distance of a border from its place, the bound, the share of the first token)"""
    row = Row(lib, x, t)
    real = real_masses(x, row.order, t)
    W, R = Decimal(int(row.upto[-1])), real[-1]
    far = max(abs(Decimal(int(a)) / W - b / R) for a, b in zip(row.upto[::7].tolist() + row.upto[-3:].tolist(), real[::7] + real[-3:]))
    return far, Decimal(2) ** -34 + len(x) * Decimal(2) ** -45, Decimal(ONE) / R


@pytest.mark.parametrize("depth", [10.0, 20.0, 23.0, 27.0, 29.0, 30.0, 31.0, 31.25])
@pytest.mark.parametrize("vocab", [5000, 60000])
def test_borders_of_flat_tails(lib, depth, vocab):
    for t in (1.0, 0.7):
        x = np.full(vocab, -depth * t, dtype=np.float32)
        x[vocab // 2] = 0
        far, bound, _ = borders(lib, x, t)
        assert far <= bound, (float(far), float(bound))


def test_borders_of_falling_tails(lib):
    rng = random.Random(2)
    for _ in range(4):
        x = np.float32([-rng.uniform(0, 33) for _ in range(9000)])
        x[17] = 0
        far, bound, _ = borders(lib, x, 1.0)
        assert far <= bound


def test_a_row_whose_borders_are_further_off_than_a_weight_s_own_error(lib):
    """Two tokens of nearly the same weight above 248,318 that weigh 0.47 units each: half of the real mass lies within the
    second token, half of the sum of the held weights at the first one's end. So 2^-35 would be no bound for a border."""
    x = np.full(248320, -31.25, dtype=np.float32)
    x[0], x[1] = 0, -2.0 ** -29
    row = Row(lib, x, 1.0)
    assert row.draw(0.5)[0] == 0
    tail = 248318 * (Decimal("-31.25")).exp()
    second = (Decimal(-2) ** -29).exp()
    real = 1 / (1 + second + tail)            # where the first token's share ends
    assert real < Decimal("0.5")              # the definition names the second token
    off = Decimal("0.5") - real
    assert Decimal(2) ** -30 < off < Decimal(2) ** -29 and off <= Decimal(2) ** -34 + 248320 * Decimal(2) ** -45


def test_a_weight_below_half_a_unit_is_none(lib):
    x = np.float32([0, -31.3, -31.0, -40])    # 2^-45 is e^-31.19
    row = Row(lib, x, 1.0)
    assert row.w.tolist() == [ONE, 1, 0, 0]
    assert row.draw(1.0)[0] == 2 and Fraction(row.draw(1.0)[1]) == ONE + 1
