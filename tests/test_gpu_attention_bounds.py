"""What a call of the attention kernels may touch when its device-side arrays
hold what they should not."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, nv
from tests.kv_oracle import Cache, attention
from tests.test_gpu_attention import bound, device_cache, offsets, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_that_fall_stay_inside_the_workspace(kv):
    """start = 0, 1000, 0, 1000, ...: the sequences' rows add up to 16 times the rows that q has. The split prompt
    kernel's partial sums must stay inside the workspace, and the status word says that something is wrong."""
    m = nv()
    batch, tokens = 32, 1000
    c = Cache([1200], 1, 64, 64, kv, seed=1)
    table = c.table.to(DEV).expand(batch, -1).contiguous()
    lens = torch.full((batch,), 1200, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, tokens] * (batch // 2) + [0], dtype=torch.int32, device=DEV)
    need = m.workspace_size(m.OP_PAGED_ATTENTION, batch, tokens, 1, 1, 64)
    room = torch.full((need + (64 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    room[:4096] = 0
    q = queries(tokens, 1, 64, 2)
    out = torch.zeros(tokens, 1, 64, dtype=torch.bfloat16, device=DEV)
    m.paged_attention(q.to(DEV), device_cache(m, c), table, lens, start=start, max_new=tokens, out=out, workspace=room[:need])
    assert m.read_device_status() == m.ERR_INVALID_ARG
    assert (room[need:] == 0x5A).all()
    assert torch.isfinite(out.float()).all()
    # the counters are back at zero, and the workspace serves an orderly call afterwards
    assert not room[:4096].any()
    ref, size = attention(c, q, [tokens])
    got = m.paged_attention(q.to(DEV), device_cache(m, c), table[:1], lens[:1], start=offsets([tokens]).to(DEV), max_new=tokens,
                            workspace=room[:need]).float().cpu().double().numpy()
    assert m.read_device_status() == 0
    assert (np.abs(got - ref) <= bound(ref, size, tokens, kv)).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("most,group", [(4, 8), (32, 1), (30, 4)])
def test_a_workspace_serves_smaller_calls(kv, most, group):
    """A verify loop: the workspace of the largest step, steps with fewer drafts on it."""
    m = nv()
    lens = [1500, 300, 77]
    c = Cache(lens, 2, 16, 128, kv, seed=2)
    dc, table = device_cache(m, c), c.table.to(DEV)
    ws = m.attention_workspace(3, most, 2 * group, 2, 128)
    for new in range(most, 0, -1 if most < 9 else -5):
        q = queries(3 * new, 2 * group, 128, new)
        ref, size = attention(c, q, [new] * 3)
        got = m.paged_attention(q.to(DEV), dc, table, torch.tensor(lens, dtype=torch.int32, device=DEV), max_new=new, workspace=ws)
        assert m.read_device_status() == 0
        assert (np.abs(got.float().cpu().double().numpy() - ref) <= bound(ref, size, new * group, kv)).all()


def test_workspaces_that_are_not_device_memory_are_refused():
    m = nv()
    cache = m.kv_cache(8, 2, 16, 64)
    table, lens = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    refs, q = torch.ones(8, dtype=torch.int32, device=DEV), torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    size = max(m.workspace_size(m.OP_PAGED_ATTENTION, 2, 1, 4, 2, 64), m.workspace_size(m.OP_KV_PAGES, 8, 2))
    calls = (lambda ws: m.paged_attention(q, cache, table, lens, workspace=ws),
             lambda ws: m.kv_reserve(table, lens, refs, 16, workspace=ws),
             lambda ws: m.kv_compact(cache, table, refs, workspace=ws))
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for call in calls:
        with pytest.raises(RuntimeError):
            call(torch.zeros(size, dtype=torch.uint8))
        for bad in (one.expand(size), torch.zeros(2 * size, dtype=torch.uint8, device=DEV)[::2]):
            with pytest.raises(ValueError):
                call(bad)
        call(torch.zeros(size, dtype=torch.uint8, device=DEV))
    assert m.read_device_status() == 0
