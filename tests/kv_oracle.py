"""Plain implementations (64 bits, CPU) of the operators on a paged key-value
cache, and random caches to run them on."""
import numpy as np
import torch

NAN_E4M3 = 0x7F


def spread(lo, hi, n, seed):
    g = np.random.default_rng(seed)
    x = g.integers(lo, hi + 1, n)
    if n > 1:
        x[0], x[-1] = lo, hi
    return [int(i) for i in x]


class Cache:
    """Pools on the CPU: everything no sequence has written is NaN. `k64`, `v64`
    give positions' values."""

    def __init__(self, lens, heads, page, dim, kv, seed, spare=3, max_pages=None, gaps=()):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.page, self.dim, self.kv, self.lens = heads, page, dim, kv, list(lens)
        held = [-(-n // page) for n in lens]
        self.max_pages = max(max(held), 1) if max_pages is None else max_pages
        self.pages = sum(held) + spare
        ids = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        n = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[n:n + h].int()
            n += h
        for b, e in gaps:
            self.table[b, e] = -1
        shape = (self.pages, heads, page, dim)
        if kv == "bf16":
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            self.v = self.k.clone()
            self.k_scale = self.v_scale = None
        else:
            self.k = torch.full(shape, NAN_E4M3, dtype=torch.uint8).view(torch.float8_e4m3fn)
            self.v = torch.full(shape, NAN_E4M3, dtype=torch.uint8).view(torch.float8_e4m3fn)
            self.k_scale = (torch.rand(heads, generator=g) + 0.5) / 64
            self.v_scale = (torch.rand(heads, generator=g) + 0.5) / 64
        for b, length in enumerate(lens):
            for e in range(held[b]):
                p, rows = int(self.table[b, e]), min(page, length - e * page)
                if p < 0:
                    continue
                for pool in (self.k, self.v):
                    x = torch.randn(heads, rows, dim, generator=g)
                    if kv == "bf16":
                        pool[p, :, :rows] = x.bfloat16()
                    else:
                        pool.view(torch.uint8)[p, :, :rows] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)

    def values(self, pool, scale, b, h):
        """[positions][dim] in 64 bits; NaN where there is no page."""
        out = np.full((self.lens[b], self.dim), np.nan)
        for e in range(-(-self.lens[b] // self.page)):
            p = int(self.table[b, e])
            if 0 <= p < self.pages:
                rows = min(self.page, self.lens[b] - e * self.page)
                x = pool[p, h, :rows].float().double().numpy()
                out[e * self.page:e * self.page + rows] = x * (1.0 if scale is None else float(scale[h]))
        return out


def attention(cache, q, news, window=0, sinks=0, scale=None):
    """(out, sum of p |v|) in 64 bits; q [T][q_heads][dim]."""
    q = q.double().numpy()
    T, heads, dim = q.shape
    group = heads // cache.heads
    scale = dim ** -0.5 if scale is None else scale
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    t = 0
    for b, n in enumerate(news):
        length = cache.lens[b]
        pos = np.arange(length - n, length)[:, None]
        j = np.arange(length)[None]
        there = np.array([0 <= int(cache.table[b, x // cache.page]) < cache.pages for x in range(length)], dtype=bool)
        ok = (j <= pos) & there[None] if length else np.zeros((n, 0), dtype=bool)
        if window:
            ok = ok & ((pos - j < window) | (j < sinks))
        for h in range(cache.heads):
            k = np.nan_to_num(cache.values(cache.k, cache.k_scale, b, h))
            v = np.nan_to_num(cache.values(cache.v, cache.v_scale, b, h))
            for x in range(h * group, (h + 1) * group):
                s = np.where(ok, (q[t:t + n, x] @ k.T) * scale, -np.inf)
                some = ok.any(1)
                if not some.any():
                    continue
                p = np.exp(s[some] - s[some].max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                rows = np.flatnonzero(some) + t
                out[rows, x] = p @ v
                size[rows, x] = p @ np.abs(v)
        t += n
    return out, size
