"""The root-mean-square norm on the GPU, against 64 bits: every output form, rows of 8 to 32768 elements, one row and many,
strided heads, streams in both types, in place, in a graph, and rows that hold zeros, infinities and NaN."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_common import nv as _nv, unpack_mma_scales
from tests.norm_oracle import REL, norm, stream

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def nv():
    return _nv()


def inputs(rows, K, seed, residual="bf16", heads=0):
    g = torch.Generator().manual_seed(seed)
    shape = (rows, heads, K) if heads else (rows, K)
    x = torch.randn(shape, generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    r = None
    if residual:
        r = torch.randn(shape, generator=g) * 3
        r[..., K // 3] *= 40
        r = r.bfloat16() if residual == "bf16" else r
    return x, w, r


def cuda(t):
    return None if t is None else t.cuda()


def check_bf16(got, y):
    # one rounding to bf16 (2^-8 of the value, 2^-134 among the smallest) of what fp32 arithmetic gives
    assert got.dtype == torch.bfloat16 and got.shape == y.shape
    d = (got.cpu().double() - y).abs()
    assert bool((d <= y.abs() * (2.0 ** -8 + 2 * REL) + 2.0 ** -133).all()), float((d / y.abs().clamp(min=1e-30)).max())


def check_e4m3(codes, scales, y):
    K = y.shape[-1]
    a = y.abs().amax(-1).reshape(-1) / 448
    a[a == 0] = 1
    s = scales.cpu().double()
    assert s.shape == a.shape and bool(((s - a).abs() <= 2 * REL * a).all())
    got = codes.cpu().double().reshape(-1, K) * s[:, None]
    y = y.reshape(-1, K)
    # a rounding to E4M3: 2^-4 of the value, half a step of 2^-9 among its subnormals
    assert bool(((got - y).abs() <= y.abs() * (2.0 ** -4 + 4 * REL) + s[:, None] * 2.0 ** -10).all())


def check_nvfp4(q, y, s_t, layout):
    rows, K = y.numel() // y.shape[-1], y.shape[-1]
    y = y.reshape(rows, K).numpy()
    st = float(q.s_t.cpu().double())
    assert abs(st - s_t) <= 2 * REL * s_t, (st, s_t)
    codes = q.codes.cpu().numpy()
    sc = q.scales.cpu().numpy()
    if layout == 1:
        cols4 = (K // 16 + 3) // 4 * 4
        full = sc.reshape(-1, cols4 // 4, 32, 4, 4)
        back = full.transpose(0, 3, 2, 1, 4).reshape(-1, cols4)
        assert not back[rows:].any() and not back[:, K // 16:].any()     # padding is zero
        sc = unpack_mma_scales(sc, rows, K)
    sb = torch.from_numpy(np.ascontiguousarray(sc)).view(torch.float8_e4m3fn).double().numpy()
    most = np.abs(y.reshape(rows, K // 16, 16)).max(-1) / 6 / st
    # the block scale: one rounding to E4M3, saturating at 448
    assert np.all(np.abs(sb - np.minimum(most, 448)) <= most * (2.0 ** -4 + 8 * REL) + 2.0 ** -10)
    values = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    v = values[np.stack((codes & 15, codes >> 4), -1).reshape(rows, K)].reshape(rows, K // 16, 16)
    den = np.where(sb > 0, sb, 1)[..., None] * st
    a = np.where(sb[..., None] > 0, y.reshape(rows, K // 16, 16) / den, 0)
    half = np.where(np.abs(a) < 2, .25, np.where(np.abs(a) < 4, .5, 1.0))
    assert np.all(np.abs(np.clip(a, -6, 6) - v) <= half + np.abs(a) * 8 * REL)


def reference(x, w, r, eps=EPS, offset=0.0):
    s = stream(x, r)
    return s, norm(s, w, eps, offset)


def run(nv, form, x, w, r, s_t=None, layout=1, **kw):
    x, w, r = cuda(x), cuda(w), cuda(r)
    if form == "bf16":
        return nv.rms_norm(x, w, EPS, residual=r, **kw)
    if form == "e4m3":
        return nv.rms_norm_e4m3(x, w, EPS, residual=r, **kw)
    return nv.rms_norm_quantize(x, w, EPS, residual=r, s_t=s_t, scale_layout=layout, **kw)


def check(form, got, s, y, residual, s_t=None, layout=1):
    got = got if isinstance(got, tuple) else (got,)
    if residual:
        assert torch.equal(got[-1].cpu(), s)
        got = got[:-1]
    if form == "bf16":
        check_bf16(got[0], y)
    elif form == "e4m3":
        check_e4m3(*got, y)
    else:
        most = float(y.abs().max()) / 2688
        check_nvfp4(got[0], y, s_t if s_t is not None else most if most > 0 else 1.0, layout)


SIZES = [(1, 8), (3, 16), (5, 64), (130, 72), (1, 128), (2000, 128), (700, 256), (33, 520), (9, 1024), (1, 1032), (700, 1040),
         (1, 5120), (17, 2048), (640, 5120), (3, 8192), (2, 8200), (2, 16384), (2, 16400), (5, 32768)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_rows(nv, rows, K, residual, form):
    x, w, r = inputs(rows, K, K + rows, residual)
    s, y = reference(x, w, r)
    check(form, run(nv, form, x, w, r), s, y, residual)


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (129, 64), (2000, 128), (33, 528), (1, 5120), (128, 1024), (700, 1040), (17, 2048), (640, 5120),
                                    (2, 16400), (3, 32768)])
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
def test_nvfp4_rows(nv, rows, K, residual, given, layout):
    x, w, r = inputs(rows, K, K + 2 * rows, residual)
    s, y = reference(x, w, r)
    s_t = 3.5 / 2688 if given else None
    t = None if s_t is None else torch.tensor([s_t], device="cuda")
    check("nvfp4", run(nv, "nvfp4", x, w, r, t, layout), s, y, residual, None if t is None else float(t.double()), layout)


@pytest.mark.parametrize("rows,K", [(64, 1024), (700, 2048)])
@pytest.mark.parametrize("given", [False, True])
def test_nvfp4_is_the_quantiser_s(nv, rows, K, given):
    """The codes are those that the quantiser gives for y, where y is not within fp32 error (2^-18) of one of the seven
    borders between codes or of a border between block scales: about 2 * 8 * 2^-18 of the elements, and 16 at once."""
    x, w, r = inputs(rows, K, 5)
    _, y = reference(x, w, r)
    st = np.float32(4.2 / 2688) if given else None
    q = run(nv, "nvfp4", x, w, r, None if st is None else torch.tensor([st], device="cuda"))[0]
    want = O.quantize(y.float().numpy(), s_t=st)
    assert (q.codes.cpu().numpy() != want.codes).mean() < 2e-3
    assert (unpack_mma_scales(q.scales.cpu().numpy(), rows, K) != want.scales).mean() < 2e-3


HEADS = [(1, 40, 16, 128), (7, 8, 4, 64), (300, 5, 2, 128), (3, 2, 1, 1040), (2, 3, 0, 16)]


@pytest.mark.parametrize("tokens,heads,others,K,form", [(*h, f) for h in HEADS for f in ("bf16", "e4m3", "nvfp4")] +
                         [(3, 2, 1, 1032, "bf16"), (3, 2, 1, 1032, "e4m3"), (2, 3, 0, 8, "bf16"), (2, 3, 0, 8, "e4m3"), (2500, 40, 3, 64, "bf16"),
                          (2500, 40, 3, 128, "e4m3"), (1300, 40, 0, 256, "nvfp4")])
def test_heads_of_a_fused_projection(nv, tokens, heads, others, K, form):
    g = torch.Generator().manual_seed(K)
    qkv = torch.randn(tokens, heads + others, K, generator=g).bfloat16()
    w = torch.randn(K, generator=g).bfloat16()
    s, y = reference(qkv[:, :heads], w, None)
    big = qkv.cuda()
    x = big[:, :heads]
    got = {"bf16": nv.rms_norm, "e4m3": nv.rms_norm_e4m3, "nvfp4": nv.rms_norm_quantize}[form](x, w.cuda(), EPS)
    check(form, got, s, y, None)
    # in place: the rest of the projection's output stays as it is
    if form == "bf16":
        assert nv.rms_norm(x, w.cuda(), EPS, out=x) is x
        check_bf16(x, y)
        assert torch.equal(big[:, heads:].cpu(), qkv[:, heads:])


@pytest.mark.parametrize("rows,K", [(1, 5120), (700, 5120), (65, 256)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_stream_in_place_and_offset_gain(nv, rows, K, kind):
    x, w, r = inputs(rows, K, 9, kind)
    w = (w.float() - 1).bfloat16()
    s, y = reference(x, w, r, offset=1.0)
    rc, xc = r.cuda(), x.cuda()
    got, out = nv.rms_norm(xc, w.cuda(), EPS, residual=rc, residual_out=rc, weight_offset=1.0, out=xc)
    assert out is rc and got is xc and torch.equal(rc.cpu(), s)
    check_bf16(xc, y)


def test_no_weight_and_other_eps(nv):
    x, _, _ = inputs(6, 384, 2, None)
    for eps in (0.0, 0.5):
        check_bf16(nv.rms_norm(x.cuda(), None, eps), norm(x, None, eps))


@pytest.mark.parametrize("K", [64, 512, 4096])
def test_values_that_are_not_ordinary(nv, K):
    """Rows of zeros, of the smallest and of large values; a NaN or an infinity stays in its row."""
    x, w, _ = inputs(8, K, 4, None)
    x[1] = 0
    x[2] = x[2] * 2.0 ** -120
    x[3] = x[3] * 2.0 ** 55
    x[5, 3] = float("nan")
    x[6, 2] = float("inf")
    y = norm(x, w, EPS)
    good = [0, 1, 2, 3, 4, 7]
    got = nv.rms_norm(x.cuda(), w.cuda(), EPS).cpu()
    check_bf16(got[good], y[good])
    assert bool(got[5].isnan().all())
    assert bool(got[6, 2].isnan()) and not got[6, 3:].any()
    codes, scales = nv.rms_norm_e4m3(x.cuda(), w.cuda(), EPS)
    check_e4m3(codes[good], scales[good], y[good])
    assert float(scales[1]) == 1.0 and not codes.view(torch.uint8)[1].cpu().any()
    assert bool(codes[5].float().isnan().all()) and bool(scales.isfinite().all())
    s_t = torch.tensor([2.0 / 2688], device="cuda")
    q = nv.rms_norm_quantize(x[good].cuda(), w.cuda(), EPS, s_t=s_t)
    check_nvfp4(q, y[good], float(s_t.double()), 1)


@pytest.mark.parametrize("K", [64, 4096])
def test_rows_next_to_the_smallest_numbers(nv, K):
    """8-bit rows whose scale would be too small to divide by: codes and scales stay finite, and near."""
    x, w, _ = inputs(6, K, 5, None)
    x = (x.float() * torch.tensor([2.0 ** -126, 2.0 ** -130, 2.0 ** -133, 2.0 ** -120, 2.0 ** -110, 0.0])[:, None]).bfloat16()
    y = norm(x, w, EPS)
    codes, scales = nv.rms_norm_e4m3(x.cuda(), w.cuda(), EPS)
    s = scales.cpu().double()
    assert bool((s >= 2.0 ** -120).all()) and float(s[5]) == 1.0
    got = codes.cpu().double() * s[:, None]
    # half a step of E4M3, and fp32's own smallest step (2^-149) in y and the products before it
    assert bool(((got - y).abs() <= y.abs() * (2.0 ** -4 + 4 * REL) + s[:, None] * 2.0 ** -10 + 2.0 ** -137).all())


def test_zeros_as_nvfp4(nv):
    q = nv.rms_norm_quantize(torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"))
    assert float(q.s_t) == 1.0 and not q.codes.any() and not q.scales.any()
    q = nv.rms_norm_quantize(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert float(q.s_t) == 1.0 and q.codes.shape == (0, 32)
    assert nv.rms_norm(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64)


def test_rows_that_do_not_start_on_16_bytes_are_copied(nv):
    x, w, _ = inputs(4, 130, 3, None)
    view = x.cuda()[:, 1:129]
    check_bf16(nv.rms_norm(view, w[:128].cuda(), EPS), norm(x[:, 1:129], w[:128], EPS))
    check_bf16(nv.rms_norm(x.cuda().t().contiguous().t()[:, :128], w[:128].cuda(), EPS), norm(x[:, :128], w[:128], EPS))


def test_neighbours_of_the_output_stay(nv):
    x, w, _ = inputs(5, 200, 3, None)
    big = torch.full((7, 208), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.rms_norm(x.cuda(), w.cuda(), EPS, out=big[1:6, :200])
    check_bf16(big[1:6, :200], norm(x, w, EPS))
    assert bool((big[0] == 7).all() and (big[6] == 7).all() and (big[:, 200:] == 7).all())


def test_refusals(nv):
    x, w, r = (cuda(t) for t in inputs(4, 64, 1))
    for bad in (dict(weight=w[:32]), dict(weight=w.float()), dict(weight=w.repeat(2)[::2]), dict(residual=r.half()), dict(residual=r[:3]),
                dict(residual=r.t().contiguous().t()), dict(residual=r, residual_out=r.float()), dict(residual=r, residual_out=r[:2]), dict(residual_out=r),
                dict(out=x[:3]), dict(out=x.float()), dict(out=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            nv.rms_norm(x, **{"weight": w, **bad})
    for bad in (dict(weight=w.cpu()), dict(residual=r.cpu()), dict(residual=r, residual_out=r.cpu()), dict(out=x.cpu())):
        with pytest.raises(RuntimeError, match="CUDA"):
            nv.rms_norm(x, **{"weight": w, **bad})
    with pytest.raises(RuntimeError, match="unsupported shape"):
        nv.rms_norm(x[:, :60].contiguous(), None)
    with pytest.raises(RuntimeError, match="unsupported shape"):
        nv.rms_norm_quantize(x[:, :56].contiguous(), None)
    with pytest.raises(RuntimeError, match="invalid argument"):
        nv.rms_norm(x, w, eps=-1.0)
    with pytest.raises(RuntimeError, match="workspace"):
        nv.rms_norm_quantize(x, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="misaligned"):
        nv.rms_norm(x, w, out=torch.empty(5 * 64, dtype=torch.bfloat16, device="cuda")[1:257].view(4, 64))
    assert torch.equal(x.cpu(), inputs(4, 64, 1)[0])


def test_in_a_graph_on_a_side_stream(nv):
    """A captured step (norm, linear, norm in 4 bits, linear) on new inputs gives what the same calls give outside."""
    rows, K, N = 5, 512, 256
    x, w, r = inputs(rows, K, 1)
    g = torch.Generator().manual_seed(2)
    wq = nv.quantize(torch.randn(K, K, generator=g).cuda() * 0.05)
    wq4 = nv.prepack_scales(nv.quantize(torch.randn(N, K, generator=g).cuda() * 0.05))
    x, w, r = x.cuda(), w.cuda(), r.cuda()
    out = torch.empty_like(r)

    def step():
        h, _ = nv.rms_norm(x, w, EPS, residual=r, residual_out=out)
        h = nv.gemm_w4a16(h, wq)
        q, s = nv.rms_norm_quantize(h, w, EPS, residual=out, residual_out=out)
        return nv.gemm_w4a4(q, wq4), s

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, s = step()
        for seed in (3, 4):
            nx, _, nr = inputs(rows, K, seed)
            x.copy_(nx)
            r.copy_(nr)
            graph.replay()
            a, b = y.clone(), s.clone()
            c, d = step()
            side.synchronize()
            assert torch.equal(a, c) and torch.equal(b, d)


def test_the_linear_behind_it(nv):
    """norm -> W4A4 linear against 64 bits on the quantised values."""
    rows, K, N = 200, 1024, 384
    x, w, r = inputs(rows, K, 6)
    wt = torch.randn(N, K, generator=torch.Generator().manual_seed(1)) * 0.05
    q, s = nv.rms_norm_quantize(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    y = nv.gemm_w4a4(q, nv.prepack_scales(nv.quantize(wt.cuda()))).float().cpu().numpy()
    _, ref = reference(x, w, r)
    want = O.gemm_w4a4(O.quantize(ref.float().numpy()), O.quantize(wt.numpy()))
    assert O.rel_fro(y, want) <= 1e-2
