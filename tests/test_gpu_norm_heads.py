"""Heads of a fused projection with a stream of their own: strided x, contiguous residual, every output form; rows that are one row of
memory, and the stream written over x."""
import pytest
import torch

from tests.gpu_common import nv as _nv
from tests.test_gpu_norm import check, check_bf16, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return _nv()


@pytest.mark.parametrize("tokens,heads,others,K", [(1, 3, 1, 128), (9, 5, 2, 64), (700, 4, 1, 128), (5, 2, 1, 1040), (650, 2, 0, 1040)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4", "nvfp4 given"])
def test_heads_with_a_residual(nv, tokens, heads, others, K, kind, form):
    g = torch.Generator().manual_seed(tokens + K)
    qkv = torch.randn(tokens, heads + others, K, generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    r = torch.randn(tokens, heads, K, generator=g).to(kind)
    s, y = reference(qkv[:, :heads], w, r)
    x, rc = qkv.cuda()[:, :heads], r.cuda()
    s_t = torch.tensor([4 / 2688], device="cuda") if form == "nvfp4 given" else None
    if form == "bf16":
        got = nv.rms_norm(x, w.cuda(), 1e-6, residual=rc, residual_out=rc)
        assert got[1] is rc
    elif form == "e4m3":
        got = nv.rms_norm_e4m3(x, w.cuda(), 1e-6, residual=rc)
    else:
        got = nv.rms_norm_quantize(x, w.cuda(), 1e-6, residual=rc, s_t=s_t)
    check(form.split()[0], got, s, y, True, None if s_t is None else float(s_t.double()))


def test_rows_that_are_one_row_of_memory(nv):
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(1, 256, generator=g).bfloat16(), torch.ones(256, dtype=torch.bfloat16)
    _, y = reference(x.expand(40, -1), w, None)
    check_bf16(nv.rms_norm(x.cuda().expand(40, -1), w.cuda(), 1e-6), y)


@pytest.mark.parametrize("rows,K", [(7, 256), (1300, 1040)])
def test_the_stream_over_x(nv, rows, K):
    g = torch.Generator().manual_seed(K)
    x, r = torch.randn(rows, K, generator=g).bfloat16(), torch.randn(rows, K, generator=g).bfloat16()
    s, y = reference(x, None, r)
    xc = x.cuda()
    got, out = nv.rms_norm(xc, None, 1e-6, residual=r.cuda(), residual_out=xc)
    assert out is xc and torch.equal(xc.cpu(), s)
    check_bf16(got, y)
