"""The norm's E4M3 codes are the quotients' of y and the row's scale, on rows of few different values, where many
quotients lie on a border between two codes."""
import numpy as np
import pytest
import torch

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
