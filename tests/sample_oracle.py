"""Plain implementation (64 bits, CPU) of the draw: counts of equal logits, cumulated."""
import math

import numpy as np


def draw(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(index or -1, probability) for one row of logits (float64) and one random number, as the definition orders them."""
    x = np.where(np.isnan(x), -math.inf, x)
    values, counts = np.unique(x[x > -math.inf] + 0.0, return_counts=True)
    values, counts = values[::-1], counts[::-1].astype(np.int64)
    if not len(values):
        return -1, 0.0
    if not t > 0:
        return int(np.flatnonzero(x == values[0])[0]), 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((values - values[0]) / t)
    w[values == values[0]] = 1.0
    w[np.isnan(w)] = 0.0
    if 0 < k < counts.sum():
        i = int(np.searchsorted(np.cumsum(counts), k))
        counts, w = counts[:i + 1].copy(), w[:i + 1]
        counts[i] -= counts.sum() - k
    if p < 1:
        mass = np.cumsum(counts * w)
        target = max(p, 0.0) * mass[-1]
        i = int(np.searchsorted(mass, target))
        before = mass[i - 1] if i else 0.0
        counts, w = counts[:i + 1].copy(), w[:i + 1]
        counts[i] = min(counts[i], max(1, math.ceil((target - before) / w[i])))
    if m > 0:
        i = max(1, int((w >= min(m, 1.0)).sum()))
        counts, w = counts[:i], w[:i]
    mass = np.cumsum(counts * w)
    u = 0.0 if not u > 0 else u
    if u >= 1:
        last = int(np.flatnonzero(w > 0)[-1])
        return int(np.flatnonzero(x == values[last])[counts[last] - 1]), float(w[last] / mass[-1])
    i = int(np.searchsorted(mass, u * mass[-1], side="right"))
    nth = int((u * mass[-1] - (mass[i - 1] if i else 0.0)) / w[i])
    return int(np.flatnonzero(x == values[i])[min(max(nth, 0), int(counts[i]) - 1)]), float(w[i] / mass[-1])
