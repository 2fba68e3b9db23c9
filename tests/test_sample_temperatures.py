"""Weights (csrc/sample_math.h, compiled for the CPU) at every temperature that fp32 has: where two logits' difference has no
fp32 value, where log2(e) / T or its second word has none, and down to the smallest logits."""
import math
import random
from decimal import Decimal, getcontext

import numpy as np
import pytest

from tests.sample_masses import ONE, build

getcontext().prec = 50
MOST = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def weigh(tmp_path_factory):
    lib = build(tmp_path_factory.mktemp("temperatures"))

    def one(ref, x, t):
        x, w = np.float32([x]), np.zeros(1, dtype=np.uint64)
        lib.weights(x.ctypes.data, 1, ref, t, w.ctypes.data)
        return int(w[0])
    return one


def f32(v):
    return float(np.float32(v))


def check(weigh, ref, x, t):
    ref, x, t = f32(ref), f32(x), f32(t)
    y = (Decimal(x) - Decimal(ref)) / Decimal(t)
    got = weigh(ref, x, t)
    if y < Decimal("-31.8"):
        assert got <= 1, (ref, x, t, got)
        return
    want = Decimal(2) ** 44 * y.exp()
    assert abs(got - want) <= want * Decimal(2) ** -35 + Decimal("0.51"), (ref, x, t, got, float(want))


def test_a_difference_that_overflows(weigh):
    for ref, x, t in ((3e38, -3e38, 3e38), (MOST, -MOST, MOST), (MOST, -MOST, 1e38), (2e38, -2e38, 4e37), (MOST, -1.0, MOST), (MOST, -MOST, 1.2e37)):
        check(weigh, ref, x, t)


@pytest.mark.parametrize("power", [-149, -140, -128, -126, -110, -65, -64, -63, -10, 10, 40, 63, 64, 65, 100, 110, 120, 125, 126, 127])
def test_weights_at_every_temperature(weigh, power):
    rng = random.Random(power)
    for _ in range(400):
        t = min(math.ldexp(rng.uniform(1, 2), power), MOST)
        t = max(f32(t), 2.0 ** -149)
        ref = max(-MOST, min(MOST, rng.uniform(-20, 20) * t))
        x = max(-MOST, min(ref, ref - rng.uniform(0, rng.choice((0.1, 3, 30))) * t))
        if f32(x) <= f32(ref):
            check(weigh, ref, x, t)


def test_large_logits_at_small_temperatures(weigh):
    for t in (2.0 ** -149, 2.0 ** -100, 2.0 ** -65, 1e-10):
        for ref in (1.0, 1e20, 3e38):
            assert weigh(f32(ref), f32(ref), t) == ONE
            assert weigh(f32(ref), float(np.nextafter(np.float32(ref), np.float32(0))), t) == 0
            assert weigh(f32(ref), -3e38, t) == 0 and weigh(f32(ref), -math.inf, t) == 0
        assert weigh(math.inf, 3e38, t) == 0 and weigh(math.inf, math.inf, t) == ONE


def test_infinite_temperature(weigh):
    assert weigh(3e38, -3e38, math.inf) == ONE and weigh(1.0, -math.inf, math.inf) == 0 and weigh(math.inf, 1.0, math.inf) == 0
