"""Appending to a paged key-value cache and keeping its pages, against plain
implementations. Everything here is exact: copies, whole numbers, and an 8-bit
rounding that is compared code by code."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_common import DEV, nv

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page,news,past", [
    (8, 128, 64, [1] * 9, list(range(60, 69))),
    (1, 64, 16, [1], [0]),
    (3, 64, 32, [5, 0, 70, 1, 0], [31, 7, 0, 63, 2]),
    (2, 128, 128, [300, 1, 129], [0, 127, 1]),
    (5, 128, 16, [3] * 70, [16] * 70),
])
def test_append(kv, heads, dim, page, news, past):
    m = nv()
    g = torch.Generator().manual_seed(1)
    T, lens = sum(news), [n + p for n, p in zip(news, past)]
    widest = max(-(-n // page) for n in lens)
    pages = len(lens) * widest + 2
    table = torch.randperm(pages, generator=g)[:len(lens) * widest].view(len(lens), widest).int()
    x = torch.randn(T, heads * dim * 3, generator=g).bfloat16()
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1e30, -1e30, 0.0, -0.0
    k, v = (x[:, heads * dim * i:heads * dim * (i + 1)].view(T, heads, dim) for i in (1, 2))
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    scale = (torch.rand(heads, generator=g) + 0.5) / 100
    cache = m.kv_cache(pages, heads, page, dim, dtype, scale.to(DEV), (scale * 0.7).to(DEV))
    for pool in (cache.k, cache.v):
        pool.view(torch.uint8).fill_(5)
    xd = x.to(DEV)
    kd, vd = (xd[:, heads * dim * i:heads * dim * (i + 1)].view(T, heads, dim) for i in (1, 2))
    uniform = min(news) == max(news)
    m.kv_append(cache, kd, vd, table.to(DEV), ints(lens), start=None if uniform else ints(np.cumsum([0] + news)),
                max_new=max(news))
    assert m.read_device_status() == 0
    for pool, rows, sc in ((cache.k, k, scale), (cache.v, v, scale * 0.7)):
        got = pool.cpu().view(torch.uint8).view(pages, heads, page, -1).numpy()
        want = np.full_like(got, 5)
        if kv == "bf16":
            codes = rows.contiguous().view(torch.uint8).view(T, heads, -1).numpy()
        else:
            y = (rows.float() / sc[:, None]).numpy().astype(np.float32)
            codes = np.where(np.signbit(y), 0x80, 0).astype(np.uint8) | O.e4m3_encode(np.abs(y)).astype(np.uint8)
        t = 0
        for b, n in enumerate(news):
            for i in range(n):
                pos = past[b] + i
                want[int(table[b, pos // page]), :, pos % page] = codes[t]
                t += 1
        assert np.array_equal(got, want)


def test_append_skips_rows_without_a_page():
    m = nv()
    cache = m.kv_cache(4, 2, 16, 64)
    for pool in (cache.k, cache.v):
        pool.zero_()
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    # no page; an id past the pool; a position past the table; a negative position
    m.kv_append(cache, x, x, ints([[-1], [4], [0], [1]]), ints([1, 2, 17, 0]))
    assert m.read_device_status() == m.ERR_INVALID_ARG
    assert not cache.k.any() and not cache.v.any()


class Pages:
    """The page bookkeeping in plain Python."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = table.copy(), lens.copy(), refs.copy(), page

    def lowest(self):
        free = np.flatnonzero(self.refs <= 0)
        return int(free[0]) if len(free) else -1

    def fork(self, src, dst, pools):
        shared = []
        for s, d in zip(src, dst):
            n, full = int(self.lens[s]), int(self.lens[s]) // self.page
            self.table[d] = -1
            self.table[d, :full] = self.table[s, :full]
            shared += [p for p in self.table[s, :full] if p >= 0]
            if n % self.page and self.table[s, full] >= 0:
                p = self.lowest()
                if p >= 0:
                    self.refs[p] = 1
                    for pool in pools:
                        pool[p, :, :n % self.page] = pool[self.table[s, full], :, :n % self.page]
                self.table[d, full] = p
            self.lens[d] = n
        for p in shared:
            self.refs[p] += 1

    def release(self, seqs):
        for b in seqs:
            for p in self.table[b][self.table[b] >= 0]:
                self.refs[p] -= 1
            self.table[b], self.lens[b] = -1, 0

    def reserve(self, news):
        for b, n in enumerate(news):
            if n:
                for e in range((self.lens[b] - n) // self.page, -(-self.lens[b] // self.page)):
                    if self.table[b, e] < 0:
                        p = self.lowest()
                        if p >= 0:
                            self.refs[p] = 1
                        self.table[b, e] = p

    def compact(self, pools):
        live = int((self.refs > 0).sum())
        src = [p for p in np.flatnonzero(self.refs > 0) if p >= live]
        dst = [p for p in np.flatnonzero(self.refs <= 0) if p < live]
        for s, d in zip(src, dst):
            for pool in pools:
                pool[d] = pool[s]
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.table[self.table == s] = d
        return live


def scattered(seed, rows, max_pages, pages, page, held):
    g = np.random.default_rng(seed)
    table = np.full((rows, max_pages), -1, dtype=np.int32)
    lens = np.zeros(rows, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    ids = iter(g.permutation(pages))
    for b, n in enumerate(held):
        lens[b] = n
        for e in range(-(-n // page)):
            table[b, e] = next(ids)
            refs[table[b, e]] = 1
    return table, lens, refs


def bits(pool):
    return pool.view(torch.int16 if pool.dtype == torch.bfloat16 else torch.uint8).cpu().numpy()


@pytest.mark.parametrize("kv,dim", [("bf16", 64), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("page,held,ways", [(16, [1], 1), (32, [33, 64, 0, 100, 7], 3), (64, [200] * 40, 4),
                                            (16, [500, 17, 16], 600)])
def test_fork_release_reserve_compact(kv, dim, page, held, ways):
    m = nv()
    heads, n = 2, len(held)
    rows, max_pages = n * (1 + ways), max(-(-x // page) for x in held) + 1
    pages = sum(-(-x // page) for x in held) + n * ways * 2 + 7
    table, lens, refs = scattered(ways, rows, max_pages, pages, page, held)
    cache = m.kv_cache(pages, heads, page, dim, torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn)
    for i, pool in enumerate((cache.k, cache.v)):
        pool.view(torch.uint8).copy_(torch.randint(0, 255, pool.view(torch.uint8).shape, dtype=torch.uint8, device=DEV,
                                                   generator=torch.Generator(device=DEV).manual_seed(i)))
    plain, pools = Pages(table, lens, refs, page), [bits(cache.k).copy(), bits(cache.v).copy()]
    # the table as a part of a wider buffer
    wide = torch.full((rows, max_pages + 3), 77, dtype=torch.int32, device=DEV)
    t, ln, r = wide[:, 1:1 + max_pages], ints(lens), ints(refs)
    t.copy_(ints(table))

    def same():
        assert np.array_equal(t.cpu().numpy(), plain.table)
        assert np.array_equal(ln.cpu().numpy(), plain.lens)
        assert np.array_equal(r.cpu().numpy(), plain.refs)
        assert np.array_equal(bits(cache.k), pools[0]) and np.array_equal(bits(cache.v), pools[1])
        assert (wide[:, 0] == 77).all() and (wide[:, 1 + max_pages:] == 77).all()
        assert m.read_device_status() == 0

    src = np.repeat(np.arange(n), ways)
    dst = n + np.random.default_rng(2).permutation(n * ways)
    m.kv_fork(cache, t, ln, r, ints(src), ints(dst))
    plain.fork(src, dst, pools)
    same()
    gone = list(range(0, n)) + [int(dst[0])]
    m.kv_release(t, ln, r, ints(gone))
    plain.release(gone)
    same()
    # every sequence grows: some within a page, some into new ones, some not at all
    news = [(3 * b) % (page + 2) for b in range(rows)]
    news = [min(x, max_pages * page - int(plain.lens[b])) for b, x in enumerate(news)]
    plain.lens += np.array(news, dtype=np.int32)
    ln.copy_(ints(plain.lens))
    m.kv_reserve(t, ln, r, page, start=ints(np.cumsum([0] + news)), max_new=max(max(news), 1))
    plain.reserve(news)
    same()
    live = m.kv_compact(cache, t, r)
    assert int(live) == plain.compact(pools)
    same()
    assert (r[:int(live)] > 0).all() and not r[int(live):].any()


@pytest.mark.parametrize("pages", [1, 15, 1000, 16384, 16385, 50001])
@pytest.mark.parametrize("used", [0.0, 0.03, 0.6, 1.0])
def test_compact_pools_of_many_sizes(pages, used):
    m = nv()
    g = np.random.default_rng(pages)
    refs = (g.random(pages) < used).astype(np.int32) * g.integers(1, 4, pages).astype(np.int32)
    table = np.full((3, pages), -1, dtype=np.int32)
    for b in range(3):
        ids = np.flatnonzero(refs > b)
        table[b, :len(ids)] = g.permutation(ids)
    cache = m.kv_cache(pages, 1, 16, 64, torch.float8_e4m3fn)
    for i, pool in enumerate((cache.k, cache.v)):
        pool.view(torch.uint8).copy_(torch.randint(0, 255, pool.view(torch.uint8).shape, dtype=torch.uint8, device=DEV))
    plain, pools = Pages(table, np.zeros(3, np.int32), refs, 16), [bits(cache.k).copy(), bits(cache.v).copy()]
    src = [p for p in np.flatnonzero(refs > 0) if p >= (refs > 0).sum()]
    moved = {s: d for s, d in zip(src, [p for p in np.flatnonzero(refs <= 0) if p < (refs > 0).sum()])}
    t, r = ints(table), ints(refs)
    live = m.kv_compact(cache, t, r)
    assert int(live) == int((refs > 0).sum())
    for s, d in moved.items():
        pools[0][d], pools[1][d] = pools[0][s], pools[1][s]
        refs[d], refs[s] = refs[s], 0
    to = np.arange(pages, dtype=np.int32)
    for s, d in moved.items():
        to[s] = d
    assert np.array_equal(t.cpu().numpy(), np.where(table >= 0, to[table], table))
    assert np.array_equal(r.cpu().numpy(), refs)
    assert np.array_equal(bits(cache.k), pools[0]) and np.array_equal(bits(cache.v), pools[1])


def test_forks_without_free_pages_and_bad_lists():
    m = nv()
    cache = m.kv_cache(3, 1, 16, 64)
    cache.k.zero_(), cache.v.zero_()
    table, lens, refs = ints([[0, 1], [-1, -1], [-1, -1], [-1, -1]]), ints([20, 0, 0, 0]), ints([1, 1, 0])
    m.kv_fork(cache, table, lens, refs, ints([0, 0]), ints([1, 2]))
    assert m.read_device_status() == m.ERR_NO_PAGES
    assert table.cpu().tolist() == [[0, 1], [0, 2], [0, -1], [-1, -1]]
    assert refs.cpu().tolist() == [3, 1, 1] and lens.cpu().tolist() == [20, 20, 20, 0]
    m.kv_fork(cache, table, lens, refs, ints([4, -1, 0]), ints([3, 3, 9]))
    assert m.read_device_status() == m.ERR_INVALID_ARG
    assert refs.cpu().tolist() == [3, 1, 1]
    m.kv_release(table, lens, refs, ints([-5, 4]))
    assert m.read_device_status() == m.ERR_INVALID_ARG
    assert refs.cpu().tolist() == [3, 1, 1]
    # reserve: one page is free for two sequences
    m.kv_release(table, lens, refs, ints([1]))
    lens.copy_(ints([20, 5, 20, 6]))
    m.kv_reserve(table, lens, refs, 16, start=ints([0, 0, 5, 5, 11]), max_new=6)
    assert m.read_device_status() == m.ERR_NO_PAGES
    assert table.cpu().tolist() == [[0, 1], [2, -1], [0, -1], [-1, -1]]
    assert refs.cpu().tolist() == [2, 1, 1]


def test_appending_and_attending_in_a_captured_graph():
    """One decode step (reserve, append, attention) captured once and replayed while the lengths grow."""
    m = nv()
    from tests.kv_oracle import Cache, attention
    B, heads, group, dim, page, steps = 3, 2, 4, 64, 16, 20
    past = [14, 0, 47]
    cache = m.kv_cache(40, heads, page, dim)
    cache.k.fill_(float("nan")), cache.v.fill_(float("nan"))
    table, lens, refs = ints(np.full((B, 8), -1)), ints(past), ints([0] * 40)
    m.kv_reserve(table, lens, refs, page, start=ints(np.cumsum([0] + past)), max_new=max(past))
    first = torch.randn(2, sum(past), heads, dim, generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    m.kv_append(cache, first[0], first[1], table, lens, start=ints(np.cumsum([0] + past)), max_new=max(past))
    x = torch.randn(steps, B, heads * (group + 2), dim, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    qkv = torch.empty_like(x[0])
    ws = m.attention_workspace(B, 1, heads * group, heads, dim)
    pws = torch.empty(m.workspace_size(m.OP_KV_PAGES, 40, B), dtype=torch.uint8, device=DEV)
    out = torch.empty(B, heads * group, dim, dtype=torch.bfloat16, device=DEV)

    def step():
        lens.add_(1)
        m.kv_reserve(table, lens, refs, page, workspace=pws)
        m.kv_append(cache, qkv[:, heads * group:heads * (group + 1)], qkv[:, heads * (group + 1):], table, lens)
        m.paged_attention(qkv[:, :heads * group], cache, table, lens, out=out, workspace=ws)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        before = [t.clone() for t in (table, lens, refs)]
        step()
        for t, b in zip((table, lens, refs), before):
            t.copy_(b)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for i in range(steps):
        qkv.copy_(x[i])
        graph.replay()
    torch.cuda.synchronize()
    assert m.read_device_status() == 0
    c = Cache([p + steps for p in past], heads, page, dim, "bf16", seed=0, max_pages=8)
    c.table, c.k, c.v, c.pages = table.cpu(), cache.k.cpu(), cache.v.cpu(), 40
    ref, size = attention(c, x[-1][:, :heads * group].cpu(), [1] * B)
    got = out.float().cpu().double().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size).all()
