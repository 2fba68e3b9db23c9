"""The norm's E4M3 codes are the quotients of y and the row's scale, and its NVFP4 codes the quantiser's, also on rows of few values, where many
quotients lie on a border between two codes."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_common import nv as _nv

F = np.float32


@pytest.fixture(scope="module")
def nv():
    return _nv()


def rows_of_borders(rows, K, seed, most=448.0):
    """Rows whose quotients are values of E4M3 and the middles between two of them, each row times a power of two."""
    g = torch.Generator().manual_seed(seed)
    steps = torch.arange(16, 32) / 16.0   # E4M3 has eight steps in an octave: every second of these is a border
    x = steps[torch.randint(0, 16, (rows, K), generator=g)] * 2.0 ** torch.randint(-5, 8, (rows, K), generator=g)
    x *= torch.where(torch.rand(rows, K, generator=g) < 0.5, -1.0, 1.0)
    x[:, 0] = most
    x *= 2.0 ** torch.randint(-20, 20, (rows, 1), generator=g)
    assert torch.equal(x.bfloat16().float(), x)
    return x


def e4m3(v):
    return torch.from_numpy(np.clip(v, F(-448), F(448))).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def candidates(x, eps):
    """(r, y, scale) for the values that fp32 arithmetic may give 1 / sqrt(mean + eps): within 8 units of it."""
    x64 = x.astype(np.float64)
    r = F(1 / np.sqrt(np.mean(x64 * x64) + float(F(eps))))
    for _ in range(8):
        r = np.nextafter(r, F(0))
    for _ in range(17):
        y = x * r
        yield y, np.abs(y).max() / F(448)
        r = np.nextafter(r, F(np.inf))


def test_the_rows_tell_products_from_quotients():
    """(Checks the inputs below: products with a rounded reciprocal give other codes on most rows.)"""
    x = rows_of_borders(40, 2048, 3).numpy()
    other = 0
    for row in x:
        y, a = list(candidates(row, 1e-6))[8]
        other += not np.array_equal(e4m3(y / a), e4m3(y * (F(1) / a)))
    assert other >= 10


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(40, 2048), (400, 64), (70, 512), (1, 5120), (3, 16392)])
@pytest.mark.parametrize("size", [0, -60, -90])   # (rows far below eps have scales far below one)
def test_codes_are_the_quotients(nv, rows, K, residual, size):
    x = rows_of_borders(rows, K, K) * 2.0 ** size
    r = None
    if residual:
        r = torch.zeros_like(x).to(torch.bfloat16 if residual == "bf16" else torch.float32).cuda()
    codes, scales = nv.rms_norm_e4m3(x.bfloat16().cuda(), None, 1e-6, residual=r)[:2]
    codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    for i, row in enumerate(x.numpy()):
        near = [(y, a) for y, a in candidates(row, 1e-6) if a == scales[i]]
        assert near, (i, scales[i])
        assert any(np.array_equal(codes[i], e4m3(y / a)) for y, a in near), i


@pytest.mark.gpu
def test_a_scale_that_overflows(nv):
    """y above the largest number: the row's scale is infinite, and finite values are 0 beside it."""
    x = torch.ones(2, 64)
    x[0, 5] = 64
    codes, scales = nv.rms_norm_e4m3(x.bfloat16().cuda(), torch.full((64,), 1e38, dtype=torch.bfloat16, device="cuda"))
    codes = codes.view(torch.uint8).cpu()
    assert float(scales[0]) == float("inf") and int(codes[0, 5]) == 0x7F and not codes[0, :5].any() and not codes[0, 6:].any()
    assert bool((codes[1] == 0x7E).all())


def ys(s, gain, eps):
    """fp32 y of one row, for the values that fp32 arithmetic may give 1 / sqrt(mean + eps) (as candidates())."""
    s64 = s.astype(np.float64)
    r = F(1 / np.sqrt(np.mean(s64 * s64) + float(F(eps))))
    for _ in range(8):
        r = np.nextafter(r, F(0))
    t = s * gain
    for _ in range(17):
        yield t * r
        r = np.nextafter(r, F(np.inf))


@pytest.mark.gpu
@pytest.mark.parametrize("borders", [False, True])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(30, 64), (20, 1024), (20, 2048), (9, 5120)])
def test_nvfp4_codes_and_scales_are_the_quantiser_s(nv, rows, K, residual, given, borders):
    """Every row's codes and block scales are those of one y that fp32 arithmetic gives."""
    g = torch.Generator().manual_seed(K)
    w = torch.ones(K) if borders else 1 + 0.2 * torch.randn(K, generator=g)
    w = w.bfloat16()
    if borders:     # few values: quotients on the borders between codes and between block scales
        x = torch.tensor([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])[torch.randint(0, 14, (rows, K), generator=g)]
        x *= 2.0 ** torch.randint(-4, 5, (rows, K // 16, 1), generator=g).repeat_interleave(16, 1).squeeze(-1)
    else:
        x = torch.randn(rows, K, generator=g)
    x = x.bfloat16()
    r = s = None
    if residual:
        r = torch.zeros(rows, K) if borders else torch.randn(rows, K, generator=g)
        r = r.to(torch.bfloat16 if residual == "bf16" else torch.float32)
        s = (x.float() + r.float()).to(r.dtype).float().numpy()
        r = r.cuda()
    else:
        s = x.float().numpy()
    s_t = torch.tensor([2.5 / 2688], device="cuda") if given else None
    q = nv.rms_norm_quantize(x.cuda(), w.cuda(), 1e-6, residual=r, s_t=s_t, scale_layout=nv.SCALES_ROWMAJOR)
    q = q[0] if residual else q
    codes, scales, st = q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.s_t.cpu().numpy()[0]
    gain = w.float().numpy()
    most = F(0)
    for i in range(rows):
        found = False
        for y in ys(s[i], gain, 1e-6):
            want = O.quantize(y[None], s_t=st)
            if np.array_equal(codes[i], want.codes[0]) and np.array_equal(scales[i], want.scales[0]):
                found, most = True, max(most, np.abs(y).max())
                break
        assert found, i
    if not given:     # of a y within the same few units
        assert abs(float(st) - float(most) / 2688) <= float(st) * 2.0 ** -19
