"""The draw's arithmetic (csrc/sample_math.h), compiled here for the CPU: keys and bins over every 16-bit value, weights
against exact decimals, products with a fraction against whole numbers."""
import ctypes
import random
import struct
import subprocess
from decimal import Decimal, getcontext
from fractions import Fraction
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parents[1] / "nvfp4_block_scaled_04_gb300" / "csrc"
getcontext().prec = 50

SOURCE = """
#include "sample_math.h"
using namespace nvfp4;
extern "C" {
unsigned key16(unsigned b) { return key_of<false>(b); }
unsigned key32(unsigned b) { return key_of<true>(b); }
float value16(unsigned k) { return value_of<false>(k); }
float value32(unsigned k) { return value_of<true>(k); }
int bin(unsigned h) { return bin_of(h); }
void range(int b, unsigned* r) { uint32_t lo, hi; bin_range(b, lo, hi); r[0] = lo; r[1] = hi; }
int sizes(int i) { return i == 0 ? NB : i == 1 ? B_MID : B_LAST; }
int wide(int b) { return wide_bin(b); }
unsigned steps(unsigned m, unsigned sign) { return bin_steps(m, sign); }
unsigned few(unsigned long long x, unsigned long long w) { return few_times(x, w); }
unsigned long long weigh(float ref, float x, float t) { return weight(ref, x, slope_of(t), EXP2_TABLE); }
unsigned long long part(unsigned long long x, float v, int* cut) { bool c = false; const unsigned long long r = times(x, v, c); *cut = c; return r; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("sample")
    (d / "m.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-shared", "-fPIC", f"-I{CSRC}", str(d / "m.cpp"), "-o", str(d / "m.so")], check=True)
    L = ctypes.CDLL(str(d / "m.so"))
    L.value16.restype = L.value32.restype = ctypes.c_float
    L.key16.restype = L.key32.restype = ctypes.c_uint
    L.weigh.restype = L.part.restype = ctypes.c_ulonglong
    L.weigh.argtypes = [ctypes.c_float] * 3
    L.few.argtypes = [ctypes.c_ulonglong] * 2
    L.few.restype = L.steps.restype = ctypes.c_uint
    L.part.argtypes = [ctypes.c_ulonglong, ctypes.c_float, ctypes.POINTER(ctypes.c_int)]
    return L


def test_keys_order_as_values(lib):
    b = np.arange(1 << 16, dtype=np.uint32)
    v = (b << 16).view(np.float32).astype(np.float64)
    k = np.array([lib.key16(int(i)) for i in b])
    there = v > -np.inf
    assert np.array_equal(k > 0, there)                      # NaN and -inf are no tokens
    order = np.argsort(v[there], kind="stable")
    kv, vv = k[there][order], v[there][order]
    assert np.array_equal(np.diff(kv) > 0, np.diff(vv) > 0) and (np.diff(kv) >= 0).all()   # -0 and 0 are one key
    for i in b[there][::97]:
        assert lib.value16(lib.key16(int(i))) == v[i]
        full = (int(i) << 16) | 0x1234
        x = struct.unpack("f", struct.pack("I", full))[0]
        if x == x:
            assert lib.value32(lib.key32(full)) == x
    assert lib.key32(0xFF800000) == 0 and lib.key32(0x7FC00000) == 0 and lib.key32(0xFFC00001) == 0
    assert lib.key32(0x80000000) == lib.key32(0) and lib.key32(0x7F800000) == 0xFF800000


def test_bins_cover_the_keys_in_falling_order(lib):
    nb, mid, last = (lib.sizes(i) for i in range(3))
    h = np.arange(0x80, 0xFF81)
    bins = np.array([lib.bin(int(i)) for i in h])
    assert (np.diff(bins) <= 0).all() and bins.min() == 0 and bins.max() == nb - 1 == last
    assert len(np.unique(bins)) == nb
    r = (ctypes.c_uint * 2)()
    for b in range(nb):
        lib.range(b, r)
        mine = h[bins == b]
        assert (r[0], r[1]) == (mine.min(), mine.max())
        assert lib.wide(b) == {0: 0, mid: 1, mid + 1: 2, last: 3}.get(b, -1)
        assert lib.wide(b) >= 0 or r[0] == r[1]
    # a bin of its own for every value of magnitude 2^-10 .. 2^7
    v = np.array([lib.value16(int(i)) for i in h])
    wide = np.isin(bins, (0, mid, mid + 1, last))
    assert np.array_equal(wide, ~((np.abs(v) >= 2.0 ** -10) & (np.abs(v) < 128)))


def test_bins_of_packed_words(lib):
    """Every bf16 of magnitude 2^-10 and more, infinities and NaN among them, in each half of a word."""
    nb, mid, last = (lib.sizes(i) for i in range(3))
    low, top = 117 << 7, 134 << 7
    for b in range(0, 1 << 16, 3):
        m, other = b & 0x7FFF, 0x4123
        if m < low:
            continue
        clamp = min(max(m, low - 1), top)
        sign = 0xFFFF if b & 0x8000 else 0
        k = lib.key16(b)
        want = lib.bin(k) if k else last if sign else 0
        for at in (0, 16):
            s = lib.steps((clamp << at) | (other << (16 - at)), sign << at)
            half = (s >> at) & 0xFFFF
            assert mid - (half - 0x10000 if half & 0x8000 else half) == want, hex(b)


def test_quotients(lib):
    rng = random.Random(5)
    for _ in range(20000):
        w = rng.randrange(1, 1 << rng.randrange(1, 45))
        n = rng.randrange(0, 1 << rng.randrange(1, 20))
        for x in (n * w, n * w + 1, max(0, n * w - 1), n * w + rng.randrange(0, w)):
            assert lib.few(x, w) == -(-x // w), (x, w)
    assert lib.few(5, 0) == 0


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


@pytest.mark.parametrize("span", [1e-4, 0.01, 1.0, 12.0, 30.0])
def test_weights(lib, span):
    """round(2^44 w) to 2^-35 of w (the sum of the roundings is 2^-36: four of 2^-25 on a term of 2^-14, two of 2^-38, 2^-33 of a
    factor of 2^-6.5, a term of 2^-39 left out) and a last rounding, never above one."""
    rng = random.Random(int(span * 1e4))
    for _ in range(3000):
        t = f32(rng.choice((1.0, 0.7, 0.6, 1.3, rng.uniform(0.05, 3))))
        ref = f32(rng.choice((rng.uniform(-20, 40), rng.uniform(-1, 1), rng.uniform(-1e-3, 1e-3), 128.5)))
        x = f32(ref - rng.uniform(0, span) * t)
        if x > ref:
            continue
        got = lib.weigh(ref, x, t)
        want = Decimal(2) ** 44 * ((Decimal(x) - Decimal(ref)) / Decimal(t)).exp()
        if x != ref and (Decimal(ref) - Decimal(x)) / Decimal(t) > Decimal("31.8"):
            assert got <= 1
            continue
        assert abs(got - want) <= want * Decimal(2) ** -35 + Decimal("0.51"), (ref, x, t, got, want)
        assert got <= 1 << 44


def test_weights_at_the_ends(lib):
    one, inf, nan = 1 << 44, float("inf"), float("nan")
    assert lib.weigh(3.0, 3.0, 0.5) == one and lib.weigh(inf, inf, 1.0) == one
    assert lib.weigh(inf, 3e38, 1.0) == 0 and lib.weigh(inf, 3.0, inf) == 0
    assert lib.weigh(3e38, -3e38, 1.0) == 0 and lib.weigh(3e38, -3e38, inf) == one
    assert lib.weigh(1.0, 0.0, inf) == one
    assert lib.weigh(1.0, 0.999, 1e-40) == 0 and lib.weigh(1.0, -100.0, 1.0) == 0
    assert abs(lib.weigh(100.0, -100.0, 1e6) - 2 ** 44 * float(Decimal("-0.0002").exp())) <= 2 ** 9


def test_parts_of_a_mass_are_exact(lib):
    rng = random.Random(3)
    cut = ctypes.c_int()
    vs = [f32(rng.random()) for _ in range(300)] + [0.5, 0.25, 2.0 ** -24, 2.0 ** -40, 2.0 ** -64, 2.0 ** -100, 1e-38, 1e-45, 1 - 2.0 ** -24, 0.0, f32(0.1)]
    for v in vs:
        for x in (1, 1 << 44, (1 << 63) - 1, rng.randrange(1, 1 << 62), 5 << 44):
            want = Fraction(v) * x
            assert lib.part(x, v, ctypes.byref(cut)) == want.numerator // want.denominator, (x, v)
            assert bool(cut.value) == (want.denominator != 1)
