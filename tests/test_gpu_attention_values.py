"""Value elements that are not finite, in every place that a cache's user can
have them: rows that do not see their token are as if they were finite, in rows
that see it their own output columns are not finite and the others stay. The
reference counts such an element as zero, so the bounds are those of
test_gpu_attention."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, nv
from tests.kv_oracle import Cache, attention
from tests.test_gpu_attention import bound, device_cache, offsets, queries

pytestmark = pytest.mark.gpu


def plant(c, places):
    """Elements (sequence, position, kv head, element) of the values; element None: all of the token's."""
    for i, (b, x, h, d) in enumerate(places):
        page, row = int(c.table[b, x // c.page]), x % c.page
        d = slice(None) if d is None else d
        if c.kv == "e4m3":
            c.v.view(torch.uint8)[page, h, row, d] = 0x7F if i % 2 else 0xFF
        else:
            c.v[page, h, row, d] = float(("nan", "inf", "-inf")[i % 3])


def seen_by(c, news, group, window, sinks, places):
    """Which outputs [T][q_heads][dim] see one of the places."""
    hit = np.zeros((sum(news), c.heads * group, c.dim), dtype=bool)
    first = np.concatenate([[0], np.cumsum(news)])
    for b, x, h, d in places:
        pos = np.arange(c.lens[b] - news[b], c.lens[b])
        sees = (x <= pos) & ((pos - x < window) | (x < sinks) if window else True)
        rows = first[b] + np.flatnonzero(sees)
        hit[rows, h * group:(h + 1) * group, slice(None) if d is None else d] = True
    return hit


def check(c, news, group, places, window=0, sinks=0, uniform=False, times=1, seed=9):
    m = nv()
    q = queries(sum(news), c.heads * group, c.dim, seed)
    plant(c, places)
    ref, size = attention(c, q, news, window, sinks)
    hit = seen_by(c, news, group, window, sinks, places)
    limit = bound(ref, size, max(news) * group, c.kv)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    args = dict(start=None if uniform else offsets(news).to(DEV), max_new=max(news), window=window, sinks=sinks,
                workspace=m.attention_workspace(len(news), max(news), c.heads * group, c.heads, c.dim))
    dc, table, qd = device_cache(m, c), c.table.to(DEV), q.to(DEV)
    for _ in range(times):
        got = m.paged_attention(qd, dc, table, lens, **args)
        assert m.read_device_status() == 0
        got = got.float().cpu().double().numpy()
        assert not np.isfinite(got[hit]).any()
        assert (np.abs(got - ref)[~hit] <= limit[~hit]).all()
    return hit


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_between_many_idle_sequences(kv):
    """A padded verify batch: 64 live sequences among 2048, the others of length 0. The copies of a live item are
    asked for many idle items before its turn; what was taken out of its values has to come back to it."""
    batch, heads, group, new, dim = 2048, 8, 2, 3, 64
    g = np.random.default_rng(3)
    live = sorted(int(b) for b in g.choice(batch, 64, replace=False))
    lens = [0] * batch
    for b in live:
        lens[b] = int(g.integers(4, 200))
    c = Cache(lens, heads, 16, dim, kv, seed=5)
    places = [(b, lens[b] - 1 - i % 2, h, (7 * b + h) % dim) for i, b in enumerate(live) for h in range(0, heads, 1 + i % 3)]
    hit = check(c, [new] * batch, group, places, uniform=True, times=5)
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_items_one_after_another(kv):
    """More items than SMs, so that one item's values are looked at while the last one's outputs are written, with
    an element in every sixteenth: no output may hold what another item remembers."""
    batch, heads, group, new, dim = 60, 8, 4, 20, 64
    c = Cache([new + 3 * b for b in range(batch)], heads, 16, dim, kv, seed=6)
    places = [(b, c.lens[b] - 1 - b % 5, (5 * b) % heads, (11 * b) % dim) for b in range(batch) if b % 2 == 0]
    hit = check(c, [new] * batch, group, places, uniform=True, times=10)
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,news,past,window,sinks", [
    (4, [4, 3], [60, 200], 0, 0),
    (1, [32, 7], [31, 500], 0, 0),          # 32 tokens of one query head in an item
    (5, [4, 4, 4], [0, 9000, 77], 0, 0),    # split over the length
    (2, [9, 12], [300, 40], 20, 3),
    (1, [32], [1000], 1, 0),
    (1, [30, 5], [700, 90], 33, 70),
])
def test_whole_rows_of_few_tokens(kv, dim, group, news, past, window, sinks):
    """A token that overflowed: all of its values. The last new one, one in the middle of the new ones, the first of a
    window, and a sink."""
    lens = [n + p for n, p in zip(news, past)]
    c = Cache(lens, 2, 16, dim, kv, seed=40 + dim)
    places = []
    for b, (n, length) in enumerate(zip(news, lens)):
        for x in {length - 1, length - n // 2, max(0, length - n + 1 - max(window, 1) // 2), max(0, length - max(window, 1))}:
            places.append((b, x, b % 2, None))
    hit = check(c, news, group, places, window, sinks)
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_every_new_token_of_a_verify_step(kv):
    """All values of all new tokens: the first row sees its own token only, and nothing reaches another head."""
    c = Cache([25, 4, 640], 3, 32, 64, kv, seed=50)
    places = [(b, c.lens[b] - i, 1, None) for b in range(3) for i in (1, 2, 3)]
    hit = check(c, [4, 4, 4], 3, places, uniform=True)
    assert not hit[:, :3].any() and not hit[:, 6:].any() and not hit[0].any() and hit[1:4, 3:6].all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,news,past,window,sinks", [
    (4, [90, 130], [0, 500], 0, 0),
    (1, [300, 257], [40, 1], 0, 0),         # 256 tokens of one query head in an item
    (4, [40], [9000], 0, 0),                # split over the positions
    (3, [200, 64], [300, 77], 100, 5),
    (1, [600, 280], [0, 513], 130, 3),
    (5, [60, 90], [300, 0], 1, 0),
    (8, [40, 33], [2000, 700], 700, 300),
])
def test_whole_rows_of_prompts(kv, dim, group, news, past, window, sinks):
    """A token that overflowed: all of its values, at the same places as for a few tokens, and one of the first."""
    lens = [n + p for n, p in zip(news, past)]
    c = Cache(lens, 2, 16, dim, kv, seed=60 + dim)
    places = []
    for b, (n, length) in enumerate(zip(news, lens)):
        for x in {length - 1, length - n // 2, max(0, length - n + 1 - max(window, 1) // 2), max(0, length - max(window, 1)), length - n + 2}:
            places.append((b, x, b % 2, None))
    hit = check(c, news, group, places, window, sinks)
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 64])
def test_every_other_new_token_of_a_prompt(kv, window):
    """Half of all new tokens' values, in a batch whose other sequences are finite: the rows before the first stay
    exact, and no sequence changes another, whatever a thread block has met before."""
    batch, new = 40, 150
    c = Cache([new + b for b in range(batch)], 4, 16, 64, kv, seed=70)
    places = [(b, c.lens[b] - 1 - i, 2, None) for b in range(0, batch, 3) for i in range(0, new - 20, 2)]
    hit = check(c, [new] * batch, 2, places, window=window, sinks=2 if window else 0, uniform=True, times=2)
    assert hit.any() and not hit.all()
