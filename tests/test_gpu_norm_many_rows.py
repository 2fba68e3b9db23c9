"""Rows so many that a CTA takes two of them in turn (8 x 152 rows and more, longer than 1024), or a warp's lanes four at a
time (32 x 152 x 256 / lanes of a row), in the forms of one pass, with rows left over and with the scales' padding behind them."""
import pytest
import torch

from tests.gpu_common import nv as _nv
from tests.test_gpu_norm import check, inputs, reference, run

pytestmark = pytest.mark.gpu
S_T = 3.5 / 2688


@pytest.fixture(scope="module")
def nv():
    return _nv()


def go(nv, form, rows, K, residual, layout=1):
    x, w, r = inputs(rows, K, K + rows, residual)
    s, y = reference(x, w, r)
    t = torch.tensor([S_T], device="cuda") if form == "nvfp4" else None
    check(form, run(nv, form, x, w, r, t, layout), s, y, residual, None if t is None else float(t.double()), layout)


@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("rows,K", [(1216, 1040), (1217, 1040), (1281, 2064), (2433, 1040), (1300, 5120), (1217, 8208)])
def test_two_rows_of_a_cta(nv, form, rows, K, residual):
    go(nv, form, rows, K, residual)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4"])
def test_long_rows(nv, form):
    go(nv, form, 1217, 16400, "f32")


@pytest.mark.parametrize("residual", [None, "f32"])
def test_padding_rows_behind_whole_cta_rows(nv, residual):
    """128 j + 1 rows: 127 rows of padding, the second rows of CTAs and first ones' alike; and scales without padding."""
    for rows in (1153, 1281, 1409):
        go(nv, "nvfp4", rows, 1056, residual)
    go(nv, "nvfp4", 1281, 1056, residual, layout=0)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("rows,K", [(155648, 16), (155701, 16), (77825, 80), (38913, 144), (39000, 256)])
@pytest.mark.parametrize("residual", [None, "bf16"])
def test_four_rows_of_a_warp_at_a_time(nv, form, rows, K, residual):
    go(nv, form, rows, K, residual)


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_four_rows_of_heads_in_a_wide_projection(nv, form):
    tokens, heads, others, K = 4000, 39, 2, 64
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(tokens, heads + others, K, generator=g).bfloat16()
    w = torch.randn(K, generator=g).bfloat16()
    s, y = reference(qkv[:, :heads], w, None)
    x = qkv.cuda()
    got = {"bf16": nv.rms_norm, "e4m3": nv.rms_norm_e4m3}[form](x[:, :heads], w.cuda(), 1e-6)
    check(form, got, s, y, None)
    if form == "bf16":
        nv.rms_norm(x[:, :heads], w.cuda(), 1e-6, out=x[:, :heads])
        check(form, x[:, :heads], s, y, None)
        assert torch.equal(x[:, heads:].cpu(), qkv[:, heads:])
