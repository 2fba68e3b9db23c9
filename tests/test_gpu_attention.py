"""Attention over a paged key-value cache against its definition in 64 bits.

Bounds. An output is rounded once to bf16: 2^-9 of it, doubled for the fp32
work before. Each weight p carries a relative error: from its score (fp32
sums of exact products, |x| below about 50 in powers of two: 2^-17) and from
its rounding for the second product, 2^-9 at most as one bf16, below 2^-16 as
two bf16 halves, 2^-11 as one f16. So |error| <= 2^-8 |out| + c sum p |v| with
c = 2^-8 where one bf16 carries p (blocks of many rows on a bf16 cache) and
c = 2^-10 elsewhere."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, nv
from tests.kv_oracle import Cache, attention, spread

pytestmark = pytest.mark.gpu


def device_cache(m, c):
    up = lambda t: None if t is None else t.to(DEV)
    return m.KVCache(up(c.k), up(c.v), up(c.k_scale), up(c.v_scale))


def offsets(news):
    return torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32)


def queries(T, heads, dim, seed):
    return (torch.randn(T, heads, dim, generator=torch.Generator().manual_seed(seed)) * 1.5).bfloat16()


def bound(ref, size, rows_of_a_head, kv):
    c = 2.0 ** -8 if kv == "bf16" and rows_of_a_head > 32 else 2.0 ** -10
    return 2.0 ** -8 * np.abs(ref) + c * size + 1e-30


def check(c, news, group, window=0, sinks=0, scale=None, uniform=False, seed=0):
    m = nv()
    T = sum(news)
    q = queries(T, c.heads * group, c.dim, seed + 77)
    ref, size = attention(c, q, news, window, sinks, scale)
    out = torch.full((T, c.heads * group, c.dim), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = m.attention_workspace(len(news), max(news), c.heads * group, c.heads, c.dim)
    args = dict(start=None if uniform else offsets(news).to(DEV), max_new=max(news), window=window, sinks=sinks,
                scale=scale, workspace=ws)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    dc = device_cache(m, c)
    m.paged_attention(q.to(DEV), dc, c.table.to(DEV), lens, out=out, **args)
    got = out.float().cpu().double().numpy()
    assert m.read_device_status() == 0
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / bound(ref, size, max(news) * group, c.kv)).max()
    assert worst <= 1.0, worst
    # the same call again, on the same workspace: the same bits, and the counters are back at zero
    again = m.paged_attention(q.to(DEV), dc, c.table.to(DEV), lens, **args)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert not ws[:4096].any()
    return got


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,page,lens", [
    (1, 1, 16, [1]),
    (2, 4, 64, [1, 2, 63, 64, 65]),
    (8, 4, 16, [1999]),
    (3, 5, 32, [700, 3, 129, 1, 1024, 333]),
    (1, 8, 128, [5000, 128, 127]),
    (2, 12, 64, [257, 600]),
    (1, 27, 32, [513]),
])
def test_one_new_token(kv, dim, heads, group, page, lens):
    c = Cache(lens, heads, page, dim, kv, seed=len(lens) + dim)
    check(c, [1] * len(lens), group, uniform=True)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group,dim,page,news,past", [
    (8, 5, 128, 16, [4] * 5, [517, 0, 64, 1000, 61]),
    (2, 3, 64, 64, [1, 0, 5, 2, 0], [100, 50, 0, 63, 0]),
    (1, 1, 128, 32, [8, 8], [120, 2000]),
    (2, 7, 64, 128, [3, 4], [126, 300]),
])
def test_a_few_new_tokens(kv, heads, group, dim, page, news, past):
    c = Cache([a + b for a, b in zip(news, past)], heads, page, dim, kv, seed=3)
    check(c, news, group)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group,dim,page,news,past", [
    (2, 4, 128, 64, [300], [0]),
    (1, 5, 128, 16, [1, 130, 257], [0, 77, 600]),
    (2, 1, 64, 32, [640, 33, 0], [0, 1000, 5]),
    (1, 3, 64, 128, [129, 127], [1, 128]),
    (1, 8, 128, 64, [513], [511]),
    (1, 9, 128, 64, [65, 20], [3, 700]),
])
def test_prompts(kv, heads, group, dim, page, news, past):
    c = Cache([a + b for a, b in zip(news, past)], heads, page, dim, kv, seed=4)
    check(c, news, group)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (128, 130), (700, 7), (5000, 64)])
@pytest.mark.parametrize("news,past", [([1, 1, 1], [0, 700, 2100]), ([4, 2], [1000, 126]), ([300, 77], [0, 900])])
def test_window_and_sinks(kv, dim, window, sinks, news, past):
    c = Cache([a + b for a, b in zip(news, past)], 2, 32, dim, kv, seed=5)
    check(c, news, 3, window=window, sinks=sinks)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,past", [([1, 1], [900, 300]), ([200, 64], [800, 300])])
def test_pages_given_up_are_not_seen(kv, news, past):
    """Entries without a page inside and outside the window; ids out of range count as none."""
    lens = [a + b for a, b in zip(news, past)]
    c = Cache(lens, 2, 32, 128, kv, seed=6, gaps=[(0, e) for e in range(1, 20)] + [(1, 0), (1, 5)])
    c.table[0, 3] = c.pages
    c.table[1, 5] = 2 ** 31 - 1
    check(c, news, 4)
    check(c, news, 4, window=300, sinks=3)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[1, 1, 1], [40, 1, 30]])
def test_rows_that_see_nothing_are_zero(kv, news):
    # lengths of zero, lengths below the number of new tokens, no page at all
    c = Cache([news[0] - 1, 0, 100], 2, 16, 64, kv, seed=7, max_pages=8)
    c.table[2] = -1
    got = check(c, news, 2)
    assert (got[0] == 0).all() and (got[news[0]:] == 0).all()


def test_a_scale_of_its_own_and_large_scores():
    c = Cache([300, 90], 2, 64, 128, "bf16", seed=8)
    check(c, [1, 1], 4, scale=0.5, uniform=True)
    check(c, [60, 70], 4, scale=0.25)


@pytest.mark.parametrize("magnitude", [1e-30, 1e30])
def test_queries_of_any_magnitude_on_an_8_bit_cache(magnitude):
    m = nv()
    c = Cache([200], 2, 16, 128, "e4m3", seed=9)
    q = (queries(1, 8, 128, 1).double() * magnitude).bfloat16()
    scale = 128 ** -0.5 / magnitude
    ref, size = attention(c, q, [1], scale=scale)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32,
                                                                                          device=DEV), scale=scale)
    got = got.float().cpu().double().numpy()
    assert (np.abs(got - ref) <= bound(ref, size, 4, "e4m3")).all()


@pytest.mark.parametrize("news", [[1, 1], [70, 90]])
def test_nan_in_a_visible_place_shows(news):
    m = nv()
    c = Cache([100, 100], 1, 16, 64, "bf16", seed=10)
    c.k[int(c.table[0, 0]), 0, 3, 5] = float("nan")
    q = queries(sum(news), 2, 64, 3)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV),
                            torch.tensor(c.lens, dtype=torch.int32, device=DEV), start=offsets(news).to(DEV),
                            max_new=max(news)).float().cpu()
    assert torch.isnan(got[:news[0]]).all() and torch.isfinite(got[news[0]:]).all()


@pytest.mark.parametrize("news", [[1, 1, 1], [5, 2, 3], [90, 40, 8]])
def test_layouts_of_the_arguments(news):
    """q as a slice of a fused projection, a wider table, strided lengths' views, another stream."""
    m = nv()
    lens = [n + p for n, p in zip(news, [300, 17, 64])]
    c = Cache(lens, 2, 16, 64, "bf16", seed=11)
    T = sum(news)
    qkv = torch.randn(T, 8 + 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    ref, size = attention(c, qkv[:, :8], news)
    wide = torch.full((3, c.max_pages + 5), 2 ** 30, dtype=torch.int32)
    wide[:, 2:2 + c.max_pages] = c.table
    dev_wide = wide.to(DEV)
    lens_d = torch.tensor([9] + lens, dtype=torch.int32, device=DEV)[1:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dc, fused, start = device_cache(m, c), qkv.to(DEV), offsets(news).to(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = m.paged_attention(fused[:, :8], dc, dev_wide[:, 2:2 + c.max_pages], lens_d, start=start, max_new=max(news))
    side.synchronize()
    got = got.float().cpu().double().numpy()
    assert (np.abs(got - ref) <= bound(ref, size, max(news) * 4, "bf16")).all()


@pytest.mark.parametrize("kv,news", [("bf16", 1), ("e4m3", 1), ("bf16", 80)])
def test_pools_past_4_gb(kv, news):
    """The pages in use are the last ones of pools of more than 2^32 bytes (and elements)."""
    m = nv()
    size = 2 if kv == "bf16" else 1
    c = Cache([700 + news], 4, 64, 128, kv, seed=12)
    page_bytes = 4 * 64 * 128 * size
    pages = (1 << 32) * 5 // 4 * size // page_bytes
    dtype = c.k.dtype
    pools = []
    for pool in (c.k, c.v):
        big = torch.empty(pages, 4, 64, 128, dtype=dtype, device=DEV)
        big[-c.pages:].view(torch.uint8).copy_(pool.view(torch.uint8))
        pools.append(big)
    up = lambda t: None if t is None else t.to(DEV)
    cache = m.KVCache(*pools, up(c.k_scale), up(c.v_scale))
    table = torch.where(c.table >= 0, c.table + (pages - c.pages), c.table)
    q = queries(news, 16, 128, 2)
    ref, a = attention(c, q, [news])
    got = m.paged_attention(q.to(DEV), cache, table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV),
                            max_new=news).float().cpu().double().numpy()
    assert (np.abs(got - ref) <= bound(ref, a, news * 4, kv)).all()


def test_many_sequences():
    c = Cache(spread(1, 60, 700, 1), 1, 16, 64, "bf16", seed=13)
    check(c, [1] * 700, 2, uniform=True)


def test_more_new_tokens_than_announced_are_computed():
    m = nv()
    c = Cache([150, 20], 1, 16, 64, "bf16", seed=14)
    news = [50, 9]
    q = queries(59, 2, 64, 5)
    ref, size = attention(c, q, news)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV),
                            torch.tensor(c.lens, dtype=torch.int32, device=DEV), start=offsets(news).to(DEV), max_new=3)
    got = got.float().cpu().double().numpy()
    assert (np.abs(got - ref) <= bound(ref, size, 6, "bf16")).all()


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[1, 1], [60, 70]])
def test_scales_that_are_not_positive(kv, news, scale):
    c = Cache([300, 90], 2, 32, 64, kv, seed=15)
    check(c, news, 4, scale=scale, window=100, sinks=2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,news", [(64, [1, 5]), (65, [1, 2]), (96, [9]), (128, [2, 3])])
def test_many_query_heads_on_one(kv, group, news):
    c = Cache([n + 200 for n in news], 1, 16, 64, kv, seed=16)
    check(c, news, group)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_short_chunk_on_a_long_context(kv):
    """Few row blocks: each is split over the positions and joined."""
    c = Cache([9000 + 40, 3000 + 33], 2, 64, 128, kv, seed=17)
    check(c, [40, 33], 4)
    check(c, [40, 33], 4, window=4000, sinks=200)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("magnitude", [1e-30, 1e30])
def test_prompt_queries_of_any_magnitude(kv, magnitude):
    m = nv()
    c = Cache([300], 2, 16, 128, kv, seed=18)
    q = (queries(100, 8, 128, 1).double() * magnitude).bfloat16()
    q[50:60] = 0
    scale = 128 ** -0.5 / magnitude
    ref, size = attention(c, q, [100], scale=scale)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32,
                                                                                          device=DEV), max_new=100, scale=scale)
    got = got.float().cpu().double().numpy()
    assert (np.abs(got - ref) <= bound(ref, size, 400, kv)).all()


def test_calls_on_two_streams_do_not_meet():
    """Two calls at once, each with its own workspace."""
    m = nv()
    sides = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i, side in enumerate(sides):
        c = Cache([4000 + i, 33], 2, 64, 128, "bf16", seed=20 + i)
        q = queries(2, 8, 128, i)
        work.append((side, c, q, device_cache(m, c), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV),
                     q.to(DEV), m.attention_workspace(2, 1, 8, 2, 128)))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (side, c, q, dc, table, lens, qd, ws) in enumerate(work):
            with torch.cuda.stream(side):
                outs[i].append(m.paged_attention(qd, dc, table, lens, workspace=ws))
    torch.cuda.synchronize()
    for (side, c, q, *_), got in zip(work, outs):
        ref, size = attention(c, q, [1, 1])
        for x in got:
            assert torch.equal(x, got[0])
        assert (np.abs(got[0].float().cpu().double().numpy() - ref) <= bound(ref, size, 4, "bf16")).all()


def test_python_refusals():
    m = nv()
    k = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    cache = m.KVCache(k, k.clone())
    table, lens = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    m.paged_attention(q, cache, table, lens)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q[0]), dict(table=table.long()), dict(lens=lens[:1]),
                dict(start=lens), dict(table=table.t()), dict(out=q.float()), dict(out=q[:1])):
        args = dict(q=q, table=table, lens=lens)
        args.update(bad)
        with pytest.raises(ValueError):
            m.paged_attention(args.pop("q"), cache, args.pop("table"), args.pop("lens"), **args)
    for bad in (dict(max_new=0), dict(window=-1), dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
                dict(q=q[:1]), dict(q=q[:, :3])):
        args = dict(q=q)
        args.update(bad)
        with pytest.raises(RuntimeError):
            m.paged_attention(args.pop("q"), cache, table, lens, **args)
    with pytest.raises(RuntimeError):
        m.paged_attention(q, cache, table.cpu(), lens)
    with pytest.raises(ValueError):
        m.KVCache(k.view(torch.uint8), k.view(torch.uint8))
    with pytest.raises(ValueError):
        m.KVCache(k[..., ::2], k[..., ::2])
    codes = torch.zeros(8, 2, 16, 64, dtype=torch.float8_e4m3fn, device=DEV)
    with pytest.raises(ValueError):
        m.KVCache(codes, codes)
    with pytest.raises(ValueError):
        m.kv_append(cache, q, q[:1], table, lens)
    with pytest.raises(ValueError):
        m.kv_fork(cache, table, lens, lens, lens[:1], lens[:1])   # one count for each page
    assert m.read_device_status() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,past,window,sinks", [([5], [300], 0, 0), ([4, 3], [40, 200], 50, 3), ([90, 130], [0, 500], 0, 0),
                                                    ([200, 64], [300, 77], 100, 5), ([40], [9000], 0, 0)])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kv, dim, news, past, window, sinks):
    """Infinite and NaN elements in new tokens' values (and in one at a window's edge): rows that do not see the
    token are as if it were finite, rows that see it carry the element's own output column away, others stay."""
    m = nv()
    lens = [a + b for a, b in zip(news, past)]
    c = Cache(lens, 2, 16, dim, kv, seed=30 + dim)
    heads, group = 2, 4
    q = queries(sum(news), heads * group, dim, 9)
    ref, size = attention(c, q, news, window, sinks)
    places = []   # (sequence, position, kv head, element)
    for b, (n, length) in enumerate(zip(news, lens)):
        for x, d in ((length - 1, 3), (length - n // 2, dim - 1), (max(0, length - n + 1 - max(window, 1) // 2), 17)):
            places.append((b, x, b % heads, d))
    for i, (b, x, h, d) in enumerate(places):
        page, row = int(c.table[b, x // 16]), x % 16
        if kv == "e4m3":
            c.v.view(torch.uint8)[page, h, row, d] = 0x7F if i % 2 else 0xFF
        else:
            c.v[page, h, row, d] = float(("inf", "-inf", "nan")[i % 3])
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                            start=offsets(news).to(DEV), max_new=max(news), window=window, sinks=sinks)
    assert m.read_device_status() == 0
    got = got.float().cpu().double().numpy()
    hit = np.zeros(got.shape, dtype=bool)
    t = 0
    for b, n in enumerate(news):
        for i in range(n):
            pos = lens[b] - n + i
            for bb, x, h, d in places:
                if bb == b and x <= pos and (not window or pos - x < window or x < sinks):
                    hit[t + i, h * group:(h + 1) * group, d] = True
        t += n
    assert hit.any() and not hit.all()
    assert not np.isfinite(got[hit]).any()
    limit = bound(ref, size, max(news) * group, kv)
    # the finite elements of these rows count as they are: the reference has the same ones
    assert (np.abs(got - ref)[~hit] <= limit[~hit]).all()
