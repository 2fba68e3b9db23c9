"""Page keeping where table entries or lists hold what they should not."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, nv
from tests.test_gpu_kv_cache import ints

pytestmark = pytest.mark.gpu


def test_reserve_takes_an_id_past_the_pool_for_no_page():
    """Such an entry holds no page, so its positions get one, and an append finds it."""
    m = nv()
    cache = m.kv_cache(6, 1, 16, 64)
    cache.k.zero_(), cache.v.zero_()
    table, lens = ints([[6, 2 ** 31 - 1, -7], [2, 1000, 7]]), ints([40, 20])
    refs = ints([0, 0, 1, 0, 0, 0])
    m.kv_reserve(table, lens, refs, 16, start=ints([0, 40, 43]), max_new=40)
    # the second sequence's new tokens are positions 17..19: entry 1 alone
    assert table.cpu().tolist() == [[0, 1, 3], [2, 4, 7]]
    assert refs.cpu().tolist() == [1, 1, 1, 1, 1, 0]
    x = torch.ones(43, 1, 64, dtype=torch.bfloat16, device=DEV)
    m.kv_append(cache, x, x, table, lens, start=ints([0, 40, 43]), max_new=40)
    assert m.read_device_status() == 0
    written = (cache.k[:, 0, :, 0] == 1).sum(1).cpu().tolist()
    assert written == [16, 16, 0, 8, 3, 0]


def test_a_source_that_is_also_a_fork_stays_inside_the_pool():
    """The lists must not do this and what the rows hold is nobody's promise, but every copy stays inside the pool:
    pages that no row names keep their contents, and every entry names a page or none."""
    m = nv()
    pages, n = 64, 12
    cache = m.kv_cache(pages, 2, 16, 64)
    for _ in range(20):
        for pool in (cache.k, cache.v):
            pool.fill_(3)
        cache.k[:2], cache.v[:2] = 1, 2
        table = torch.full((n + 1, 4), -1, dtype=torch.int32, device=DEV)
        table[0, :2] = ints([0, 1])
        lens, refs = ints([25] + [21] * n), torch.zeros(pages, dtype=torch.int32, device=DEV)
        refs[:2] = 1
        m.kv_fork(cache, table, lens, refs, ints(range(n)), ints(range(1, n + 1)))
        t, r = table.cpu().numpy(), refs.cpu().numpy()
        assert m.read_device_status() == 0
        assert ((t >= -1) & (t < pages)).all()
        free = r == 0
        assert free.sum() >= pages - 2 - n and not np.isin(np.flatnonzero(free), t).any()
        assert (cache.k[torch.from_numpy(free).to(DEV)] == 3).all() and (cache.v[torch.from_numpy(free).to(DEV)] == 3).all()
