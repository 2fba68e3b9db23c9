"""Sizes of the paged key-value cache's workspaces: one made for a call serves every smaller call."""
import pytest

from tests.test_abi import nv  # noqa: F401  (the built library)


def size(m, batch=4, max_new=1, group=1, kv_heads=2, dim=128):
    return m.workspace_size(m.OP_PAGED_ATTENTION, batch, max_new, group * kv_heads, kv_heads, dim)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 12, 16, 27, 64, 65, 128])
def test_attention_workspace_never_falls(nv, group):  # noqa: F811
    news = [*range(1, 70), 100, 1000, 8192, 1 << 20]
    for kv_heads in (1, 8):
        for dim in (64, 128):
            sizes = [size(nv, max_new=n, group=group, kv_heads=kv_heads, dim=dim) for n in news]
            assert sizes == sorted(sizes), [n for n, a, b in zip(news[1:], sizes, sizes[1:]) if b < a]
    for n in (1, 3, 40):
        assert size(nv, max_new=n, group=group, dim=64) <= size(nv, max_new=n, group=group, dim=128)
        batches = [size(nv, batch=b, max_new=n, group=group) for b in (1, 2, 64, 4096)]
        assert batches == sorted(batches)


@pytest.mark.parametrize("max_new", [1, 2, 3, 4, 5, 11, 33, 200])
def test_attention_workspace_never_falls_with_the_query_heads(nv, max_new):  # noqa: F811
    sizes = [size(nv, max_new=max_new, group=g) for g in range(1, 129)]
    assert sizes == sorted(sizes)


def test_rows_that_31_bits_do_not_count_are_refused(nv):  # noqa: F811
    from tests.test_kv_abi import P, attend, seqs
    assert attend(nv, tokens=(1 << 30) - 1, s=seqs(nv, start=P)) == -2        # 4 query heads on one
    assert attend(nv, tokens=(1 << 24) - 1, heads=8 * 128, q_stride=8 * 128 * 128, s=seqs(nv, start=P)) == -2
