"""Attention where one token outweighs all others by many powers of two: what the
light ones carry alone must still arrive.

Bounds: those of test_gpu_attention, and for E4M3 caches, whose weights are f16
with the heaviest seen so far between 2^11 and 2^15, half of f16's smallest
spacing for each token: 2^-25 of a sum of 2^11 or more, so 2^-36 sum |v|."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, nv
from tests.kv_oracle import Cache, attention
from tests.test_gpu_attention import bound, device_cache, queries

pytestmark = pytest.mark.gpu


def run(kv, dim, length, news, gap, strong, window=0, sinks=0):
    m = nv()
    group, page = 2, 128
    c = Cache([length], 1, page, dim, kv, seed=dim + gap)
    q = queries(news, group, dim, 3) / 8
    scale = dim ** -0.5
    # element 0 of the keys: 448 codes (7 without codes) in one token, zero elsewhere; queries that make it `gap` powers of two
    top = 448 * float(c.k_scale[0]) if kv == "e4m3" else 7.0
    q[:, :, 0] = gap * float(np.log(2.0)) / (scale * top)
    q = q.bfloat16()
    n_pages = -(-length // page)
    ids = c.table[0, :n_pages].long()
    one = torch.tensor(448.0 if kv == "e4m3" else 7.0).to(c.k.dtype)
    raw = (lambda t: t.view(torch.uint8)) if kv == "e4m3" else (lambda t: t)
    raw(c.k)[ids, :, :, 0] = 0
    raw(c.k)[c.table[0, strong // page].long(), 0, strong % page, 0] = raw(one.reshape(1))[0]
    # light tokens' values are positive; the heavy one has nothing in the upper half
    if kv == "e4m3":
        c.v.view(torch.uint8)[ids] &= 0x7F
    else:
        c.v[ids] = c.v[ids].abs()
    raw(c.v)[c.table[0, strong // page].long(), 0, strong % page, dim // 2:] = 0
    # what lies behind the length stays NaN
    tail = length % page
    if tail:
        if kv == "e4m3":
            c.v.view(torch.uint8)[ids[-1], :, tail:] = 0x7F
            c.k.view(torch.uint8)[ids[-1], :, tail:] = 0x7F
        else:
            c.v[ids[-1], :, tail:] = float("nan")
            c.k[ids[-1], :, tail:] = float("nan")
    ref, size = attention(c, q, [news], window, sinks, scale)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor([length], dtype=torch.int32, device=DEV),
                            max_new=news, window=window, sinks=sinks).float().cpu().double().numpy()
    limit = bound(ref, size, news * group, kv)
    if kv == "e4m3":
        v = c.values(c.v, c.v_scale, 0, 0)
        limit = limit + 2.0 ** -36 * np.abs(v).sum(0)
    assert (ref[..., dim // 2:] > 0).all()
    worst = (np.abs(got - ref) / limit).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [14, 20, 25, 30])
@pytest.mark.parametrize("length,strong", [(16, 0), (16, 9), (2000, 3)])
def test_tokens(kv, dim, gap, length, strong):
    run(kv, dim, length, 1, gap, strong)
    run(kv, dim, length, 4, gap, strong)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [14, 20, 25, 30])
def test_prompts(kv, dim, gap):
    run(kv, dim, 300, 60, gap, 3)
    run(kv, dim, 1500, 200, gap, 700)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 40])
def test_a_sink_in_a_long_context(kv, news):
    """The first token against 131 thousand light ones, which hold 0.4% of the weight together; and under a window."""
    run(kv, 64, 131072, news, 25, 0)
    run(kv, 64, 131072, news, 16, 0, window=65536, sinks=1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 4, 60])
def test_a_key_that_is_not_a_number_shows(kv, news):
    """Every row that sees the key is NaN, the rows of another sequence are not."""
    m = nv()
    c = Cache([100, 100], 1, 16, 64, kv, seed=31)
    place = (int(c.table[0, 1]), 0, 3, 5)
    if kv == "e4m3":
        c.k.view(torch.uint8)[place] = 0x7F
    else:
        c.k[place] = float("nan")
    q = queries(2 * news, 2, 64, 3)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV),
                            max_new=news).float().cpu()
    assert torch.isnan(got[:news]).all() and torch.isfinite(got[news:]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 70])
@pytest.mark.parametrize("scale", [30.0, 3000.0])
def test_large_scores(kv, news, scale):
    """Scores of hundreds to a hundred thousand powers of two: one token takes nearly all. A score of 2^17 is off by
    about 2^-8 of a power of two, which moves 2^-8 of a weight between two tokens that come close."""
    m = nv()
    c = Cache([400], 2, 32, 64, kv, seed=32)
    q = queries(news, 4, 64, 8)
    ref, size = attention(c, q, [news], scale=scale)
    got = m.paged_attention(q.to(DEV), device_cache(m, c), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV),
                            max_new=news, scale=scale).float().cpu().double().numpy()
    slack = 2.0 ** -7 * size
    assert (np.abs(got - ref) <= bound(ref, size, news * 2, kv) + slack).all()
