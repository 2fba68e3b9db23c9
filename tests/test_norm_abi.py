"""CPU-side checks of the norm's C ABI and Python calls: every refusal comes back before anything is launched."""
import pytest
import torch

from tests.test_abi import nv  # noqa: F401  (the built library)

P = 0x100000   # an aligned address that is never read


def rows(m, **kw):
    a = dict(x=P, weight=P, residual=None, residual_out=None, tokens=4, x_stride=128, heads=1, K=128, residual_dtype=m.DTYPE_BF16, eps=1e-6,
             weight_offset=0.0, reserved=0)
    a.update(kw)
    return m.CNorm(*(a[f] for f, _ in m.CNorm._fields_))


NAN, INF = float("nan"), float("inf")
BAD = [(dict(x=None), -1), (dict(tokens=-1), -1), (dict(heads=0), -1), (dict(K=0), -1), (dict(reserved=1), -1), (dict(eps=-1e-6), -1), (dict(eps=NAN), -1),
       (dict(eps=INF), -1), (dict(weight_offset=NAN), -1), (dict(weight_offset=INF), -1), (dict(residual=P), -1), (dict(residual_out=P), -1),
       (dict(residual=P, residual_out=P, residual_dtype=2), -1), (dict(x_stride=127), -1), (dict(heads=2, x_stride=248), -1),
       (dict(K=100, x_stride=104), -2), (dict(K=32784, x_stride=32784), -2), (dict(tokens=(1 << 30) + 1), -2),
       (dict(tokens=1 << 20, heads=1 << 11, x_stride=1 << 18), -2), (dict(x=P + 2), -3), (dict(weight=P + 8), -3), (dict(x_stride=132), -3),
       (dict(residual=P + 4, residual_out=P), -3), (dict(residual=P, residual_out=P + 8), -3)]


@pytest.mark.parametrize("kw,code", BAD)
def test_bad_rows(nv, kw, code):  # noqa: F811
    n, L = rows(nv, **kw), nv.lib()
    assert L.nvfp4_rms_norm(n, P, 1 << 20, None) == code
    assert L.nvfp4_rms_norm_e4m3(n, P, P, None) == code
    assert L.nvfp4_rms_norm_quantize(n, P, P, P, nv.ST_COMPUTE, nv.SCALES_MMA, P, 1 << 40, None) == code


def test_bad_outputs(nv):  # noqa: F811
    n, L = rows(nv), nv.lib()
    assert L.nvfp4_rms_norm(n, None, 128, None) == -1 and L.nvfp4_rms_norm(n, P, 120, None) == -1
    assert L.nvfp4_rms_norm(n, P + 2, 128, None) == -3 and L.nvfp4_rms_norm(n, P, 132, None) == -3
    assert L.nvfp4_rms_norm_e4m3(n, None, P, None) == -1 and L.nvfp4_rms_norm_e4m3(n, P, None, None) == -1
    assert L.nvfp4_rms_norm_e4m3(n, P + 8, P, None) == -3

    def quant(n=n, codes=P, scales=P, s_t=P, mode=0, layout=1, ws=P, size=1 << 20):
        return L.nvfp4_rms_norm_quantize(n, codes, scales, s_t, mode, layout, ws, size, None)

    assert quant(codes=None) == -1 and quant(scales=None) == -1 and quant(s_t=None) == -1 and quant(mode=2) == -1 and quant(layout=2) == -1
    assert quant(codes=P + 8) == -3 and quant(ws=P + 4) == -3
    assert quant(ws=None) == -5 and quant(size=nv.workspace_size(nv.OP_RMS_NORM_QUANTIZE, 4) - 1) == -5
    assert quant(n=rows(nv, K=136, x_stride=136)) == -2     # blocks of 16
    # no rows: nothing to do, and nothing is needed
    none = rows(nv, tokens=0, x=None)
    assert L.nvfp4_rms_norm(none, None, 0, None) == 0 and L.nvfp4_rms_norm_e4m3(none, None, None, None) == 0
    assert quant(n=none, codes=None, scales=None, mode=1, ws=None, size=0) == 0


def test_workspace_grows_with_the_rows(nv):  # noqa: F811
    sizes = [nv.workspace_size(nv.OP_RMS_NORM_QUANTIZE, n) for n in (0, 1, 100, 8192)]
    assert sizes == sorted(sizes) and sizes[-1] >= sizes[0] + 4 * 8192


def test_python_refusals(nv):  # noqa: F811
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for call in (nv.rms_norm, nv.rms_norm_e4m3, nv.rms_norm_quantize):
        with pytest.raises(RuntimeError, match="CUDA"):
            call(x, w)
        with pytest.raises(ValueError, match="bf16"):
            call(x.float(), w)
        with pytest.raises(ValueError, match="rows"):
            call(x[0], w)
