"""CPU-side checks of the paged key-value cache's C ABI and Python calls: every
refusal comes back before anything is launched."""
import ctypes

import pytest
import torch

from tests.test_abi import nv  # noqa: F401  (the built library)

P = 0x100000   # an aligned address that is never read


def cache(m, **kw):
    a = dict(k=P, v=2 * P, k_scale=None, v_scale=None, pages=64, heads=8, page_size=64, head_dim=128, dtype=m.DTYPE_BF16)
    a.update(kw)
    return m.CKVCache(*(a[f] for f, _ in m.CKVCache._fields_))


def seqs(m, **kw):
    a = dict(table=P, lens=P, start=None, table_stride=16, batch=4, max_pages=16, max_new=1, reserved=0)
    a.update(kw)
    return m.CKVSeqs(*(a[f] for f, _ in m.CKVSeqs._fields_))


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(pages=0), -1), (dict(heads=0), -1),
              (dict(dtype=0), -1), (dict(dtype=2), -1), (dict(dtype=2, k_scale=P), -1), (dict(page_size=8), -2), (dict(page_size=48), -2),
              (dict(page_size=256), -2), (dict(head_dim=96), -2), (dict(head_dim=256), -2), (dict(heads=2048), -2),
              (dict(pages=1 << 28), -2), (dict(k=P + 8), -3), (dict(v=P + 2), -3)]
BAD_SEQS = [(dict(table=None), -1), (dict(lens=None), -1), (dict(batch=0), -1), (dict(max_new=0), -1), (dict(max_pages=-1), -1),
            (dict(table_stride=15), -1), (dict(reserved=1), -1), (dict(batch=5000, start=P), -2), (dict(batch=3), -1)]


def attend(m, q=P, q_stride=4096, heads=32, c=None, s=None, tokens=4, window=0, sinks=0, scale=0.1, out=P, ws=P, size=1 << 30):
    return m.lib().nvfp4_paged_attention(q, q_stride, heads, c or cache(m), s or seqs(m), tokens, window, sinks, scale, out, ws, size, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(nv, kw, code):  # noqa: F811
    c = cache(nv, **kw)
    assert attend(nv, c=c, q_stride=1 << 20, heads=2048) == code
    assert nv.lib().nvfp4_kv_append(c, seqs(nv), P, 1 << 20, P, 1 << 20, 4, None) == code
    assert nv.lib().nvfp4_kv_fork(c, P, 16, 16, P, 8, P, P, P, 2, None) == code
    assert nv.lib().nvfp4_kv_compact(c, P, 16, 16, 8, P, P, P, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", BAD_SEQS)
def test_bad_sequences(nv, kw, code):  # noqa: F811
    s = seqs(nv, **kw)
    assert attend(nv, s=s) == code
    assert nv.lib().nvfp4_kv_append(cache(nv), s, P, 1024, P, 1024, 4, None) == code
    assert nv.lib().nvfp4_kv_reserve(s, 4, 64, s.table or 0, P, 64, P, 1 << 20, None) == code


def test_bad_attention_arguments(nv):  # noqa: F811
    assert attend(nv, q=None) == -1 and attend(nv, out=None) == -1
    assert attend(nv, heads=0) == -1 and attend(nv, heads=12) == -1 and attend(nv, heads=-8) == -1
    assert attend(nv, heads=8 * 129, q_stride=8 * 129 * 128) == -2      # more query heads per kv head than the kernels take
    assert attend(nv, q_stride=4095) == -1 and attend(nv, q_stride=4097) == -3
    assert attend(nv, q=P + 2) == -3 and attend(nv, out=P + 8) == -3 and attend(nv, ws=P + 4) == -3
    assert attend(nv, window=-1) == -1 and attend(nv, sinks=-1) == -1
    assert attend(nv, scale=float("nan")) == -1 and attend(nv, scale=float("inf")) == -1
    assert attend(nv, tokens=-1) == -1 and attend(nv, tokens=5) == -1
    assert attend(nv, tokens=1 << 30, s=seqs(nv, start=P)) == -2
    need = nv.workspace_size(nv.OP_PAGED_ATTENTION, 4, 1, 32, 8, 128)
    assert need > 4096 and attend(nv, ws=None) == -5 and attend(nv, size=need - 1) == -5
    assert attend(nv, tokens=0, s=seqs(nv, start=P), q=None, out=None, ws=None, size=0) == 0   # nothing to do


def test_bad_append_arguments(nv):  # noqa: F811
    def append(k=P, ks=1024, v=P, vs=1024, tokens=4):
        return nv.lib().nvfp4_kv_append(cache(nv), seqs(nv), k, ks, v, vs, tokens, None)
    assert append(k=None) == -1 and append(v=None) == -1 and append(ks=1023) == -1 and append(vs=1016) == -1
    assert append(k=P + 2) == -3 and append(v=P + 8) == -3 and append(ks=1028) == -3 and append(vs=1025) == -3


def test_bad_page_arguments(nv):  # noqa: F811
    L, c = nv.lib(), cache(nv)
    assert L.nvfp4_kv_fork(c, None, 16, 16, P, 8, P, P, P, 2, None) == -1
    assert L.nvfp4_kv_fork(c, P, 15, 16, P, 8, P, P, P, 2, None) == -1
    assert L.nvfp4_kv_fork(c, P, 16, 16, None, 8, P, P, P, 2, None) == -1
    assert L.nvfp4_kv_fork(c, P, 16, 16, P, 8, None, P, P, 2, None) == -1
    assert L.nvfp4_kv_fork(c, P, 16, 16, P, 8, P, None, P, 2, None) == -1
    assert L.nvfp4_kv_fork(c, P, 16, 16, P, 8, P, P, P, -1, None) == -1
    assert L.nvfp4_kv_fork(c, P, 16, 16, P, 8, P, None, None, 0, None) == 0
    assert L.nvfp4_kv_release(P, 16, 16, P, 8, P, 0, P, 2, None) == -1
    assert L.nvfp4_kv_release(P, 16, 16, None, 8, P, 64, P, 2, None) == -1
    assert L.nvfp4_kv_release(P, 16, 16, P, 8, P, 64, None, 2, None) == -1
    assert L.nvfp4_kv_release(P, 16, 16, P, 8, P, 64, None, 0, None) == 0
    need = nv.workspace_size(nv.OP_KV_PAGES, 64, 0)
    assert need >= 2 * 4 * 64
    assert L.nvfp4_kv_compact(c, P, 16, 16, 8, P, None, P, need, None) == -1
    assert L.nvfp4_kv_compact(c, P, 16, 16, 8, None, P, P, need, None) == -1
    assert L.nvfp4_kv_compact(c, P, 16, 16, 8, P, P, None, need, None) == -5
    assert L.nvfp4_kv_compact(c, P, 16, 16, 8, P, P, P, need - 1, None) == -5
    assert L.nvfp4_kv_compact(c, P, 16, 16, 8, P, P, P + 4, need, None) == -3
    s = seqs(nv)
    assert L.nvfp4_kv_reserve(s, 4, 0, P, P, 64, P, 1 << 20, None) == -1
    assert L.nvfp4_kv_reserve(s, 4, 64, 2 * P, P, 64, P, 1 << 20, None) == -1     # another table than the sequences'
    assert L.nvfp4_kv_reserve(s, 4, 64, P, None, 64, P, 1 << 20, None) == -1
    assert L.nvfp4_kv_reserve(s, 4, 64, P, P, 64, P, 8, None) == -5


def test_status_and_sizes(nv):  # noqa: F811
    assert "page" in nv.lib().nvfp4_status_string(nv.ERR_NO_PAGES).decode()
    assert nv.workspace_size(nv.OP_PAGED_ATTENTION, 0, 1, 32, 8, 128) == 0
    assert nv.workspace_size(nv.OP_PAGED_ATTENTION, 1, 64, 32, 8, 128) > nv.workspace_size(nv.OP_PAGED_ATTENTION, 1, 1, 32, 8, 128)
    assert ctypes.sizeof(nv.CKVCache) == 56 and ctypes.sizeof(nv.CKVSeqs) == 48


def test_python_calls_refuse_cpu_tensors(nv):  # noqa: F811
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        nv.KVCache(k, k)
    with pytest.raises(ValueError):
        nv.KVCache(k, k[:, :, :8])
    with pytest.raises(ValueError):
        nv.KVCache(k.float(), k)
