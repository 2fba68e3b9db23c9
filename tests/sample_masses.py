"""The draw in whole numbers (CPU): weights as csrc/sample_math.h rounds them, masses added exactly, the definition's order.
What the kernel computes has to be this, whatever the logits' type and however many CTAs take a row."""
import ctypes
import subprocess
from fractions import Fraction
from pathlib import Path

import numpy as np

CSRC = Path(__file__).resolve().parents[1] / "nvfp4_block_scaled_04_gb300" / "csrc"
ONE = 1 << 44

SOURCE = """
#include "sample_math.h"
using namespace nvfp4;
extern "C" void weights(const float* x, long n, float ref, float t, unsigned long long* w) {
  const Slope c = slope_of(t);
  for (long i = 0; i < n; ++i) w[i] = weight(ref, x[i], c, EXP2_TABLE);
}
"""


def build(folder):
    (folder / "w.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-shared", "-fPIC", f"-I{CSRC}", str(folder / "w.cpp"), "-o", str(folder / "w.so")],
                   check=True)
    lib = ctypes.CDLL(str(folder / "w.so"))
    lib.weights.argtypes = [ctypes.c_void_p, ctypes.c_long, ctypes.c_float, ctypes.c_float, ctypes.c_void_p]
    return lib


def part(v, mass):
    return Fraction(float(v)) * mass


class Row:
    """A row's tokens in order, with their masses."""

    def __init__(self, lib, x, t):
        x = np.ascontiguousarray(x, dtype=np.float32) + np.float32(0)
        there = np.flatnonzero(x > -np.inf)
        self.order = there[np.argsort(-x[there].astype(np.float64), kind="stable")]
        v = np.ascontiguousarray(x[self.order])
        self.w = np.empty(len(v), dtype=np.uint64)
        lib.weights(v.ctypes.data, len(v), float(v[0]), float(np.float32(t)), self.w.ctypes.data)
        self.upto = np.cumsum(self.w)

    def draw(self, u, k=0, p=1.0, m=0.0):
        """The token, and the mass kept."""
        n, upto = len(self.w), self.upto
        if 0 < k < n:
            n = k
        if float(np.float32(p)) < 1:
            want = max(1, -(-part(np.float32(p), int(upto[n - 1])) // 1))
            n = int(np.searchsorted(upto[:n], np.uint64(want))) + 1
        if m > 0:
            least = max(1, -(-part(np.float32(m), ONE) // 1))
            n = max(1, int((self.w[:n] >= np.uint64(least)).sum()))
        W = int(upto[n - 1])
        past = W - 1 if u >= 1 else int(part(u, W))
        return int(self.order[int(np.searchsorted(upto[:n], np.uint64(past), side="right"))]), W
