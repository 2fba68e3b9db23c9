"""The draw on the GPU against 64 bits: every token has to be the one that the definition names."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import nv as _nv
from tests.sample_oracle import draw

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def nv():
    return _nv()


def logits(rows, vocab, dtype, seed, sigma=3.0, shift=4.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * sigma + shift).to(dtype)


def uniform(rows, seed):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed + 1000))


def column(v, rows, dtype):
    return torch.full((rows,), v, dtype=dtype) if not torch.is_tensor(v) else v


def check(nv, x, u, t=1.0, k=0, p=1.0, m=0.0, tensors=True, device_x=None):
    """Draws of all rows, and the same by the definition."""
    rows = x.shape[0]
    t, p, m = (column(v, rows, torch.float32) for v in (t, p, m))
    k = column(k, rows, torch.int32)
    if tensors:
        settings = (t.cuda(), k.cuda(), p.cuda(), m.cuda())
    else:
        settings = (float(t[0]), int(k[0]), float(p[0]), float(m[0]))
    ids, probs = nv.sample(x.cuda() if device_x is None else device_x, u.cuda(), *settings)
    ids, probs = ids.cpu(), probs.cpu()
    x64 = x.double().numpy()
    for r in range(rows):
        i, q = draw(x64[r], float(u[r]), float(t[r]), int(k[r]), float(p[r]), float(m[r]))
        assert int(ids[r]) == i, (r, int(ids[r]), i, float(u[r]), float(t[r]), int(k[r]), float(p[r]), float(m[r]))
        # two conversions and a division in fp32
        assert abs(float(probs[r]) - q) <= q * 2.0 ** -22, (r, float(probs[r]), q)
    return ids


MODES = {"plain": {}, "k": dict(k=20), "p": dict(p=0.8), "m": dict(m=0.05), "all": dict(t=0.7, k=50, p=0.9, m=0.02), "greedy": dict(t=0.0)}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 2), (3, 7), (5, 8), (5, 9), (40, 100), (7, 1000), (3, 4097), (160, 513), (20, 32003), (1, 151937), (2, 248320)])
def test_draws(nv, rows, vocab, dtype, mode):
    for seed in range(3 if vocab < 100000 else 2):
        check(nv, logits(rows, vocab, dtype, seed), uniform(rows, seed), **MODES[mode])


@pytest.mark.parametrize("dtype", TYPES)
def test_largest_vocabulary(nv, dtype):
    check(nv, logits(2, 524288, dtype, 3), uniform(2, 3), p=0.99)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw", [{}, dict(k=300, p=0.9), dict(t=0.0), dict(m=1e-4)])
def test_largest_vocabulary_in_one_cta(nv, dtype, kw):
    """More rows than SMs: a CTA walks the whole row (all rows are one row of memory)."""
    rows = 200
    x, u = logits(1, 524288, dtype, 13), uniform(rows, 13)
    t, k, p, m = kw.get("t", 1.0), kw.get("k", 0), kw.get("p", 1.0), kw.get("m", 0.0)
    ids, probs = nv.sample(x.cuda().expand(rows, -1), u.cuda(), t, k, p, m)
    f = lambda v: float(torch.tensor(v))   # (settings are fp32)
    for r in range(0, rows, 29):
        i, q = draw(x[0].double().numpy(), float(u[r]), f(t), k, f(p), f(m))
        assert int(ids[r]) == i and abs(float(probs[r]) - q) <= q * 2.0 ** -22


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_with_settings_of_their_own(nv, dtype):
    rows, vocab = 90, 5000
    g = torch.Generator().manual_seed(1)
    x = logits(rows, vocab, dtype, 5)
    t = torch.where(torch.arange(rows) % 7 == 0, 0.0, 0.3 + 2 * torch.rand(rows, generator=g))
    k = torch.where(torch.arange(rows) % 3 == 0, 0, torch.randint(1, 6000, (rows,), generator=g)).int()
    p = torch.where(torch.arange(rows) % 2 == 0, 1.0, torch.rand(rows, generator=g))
    m = torch.where(torch.arange(rows) % 5 < 3, 0.0, 0.3 * torch.rand(rows, generator=g))
    check(nv, x, uniform(rows, 2), t, k, p, m)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [1e-30, 1e-3, 0.004, 0.05, 0.3, 1.0, 4.0, 50.0, 1e4, 1e30, math.inf])
def test_temperatures(nv, dtype, t):
    x = logits(6, 3000, dtype, 7)
    for kw in ({}, dict(p=0.7), dict(k=100, m=0.3)):
        check(nv, x, uniform(6, 8), t=t, **kw, tensors=False)


def special(kind, rows, vocab, dtype, seed):
    x = logits(rows, vocab, torch.float32, seed)
    g = torch.Generator().manual_seed(seed)
    if kind == "equal":
        x[:] = 2.5
    elif kind == "zeros":
        x[:] = torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, -0.0)
    elif kind == "two values":
        x = torch.where(torch.rand(x.shape, generator=g) < 0.3, 1.0, -0.5)
    elif kind == "tiny":
        x *= 1e-5
    elif kind == "tiny, one ahead":
        x *= 1e-5
        x[:, vocab // 2] = 0.02
    elif kind == "padded":          # a padded vocabulary's columns are zero
        x[:, vocab // 2:] = 0
    elif kind == "padded with both zeros":
        x[:, vocab // 3:] = torch.where(torch.rand(rows, vocab - vocab // 3, generator=g) < 0.5, 0.0, -0.0)
        x[:, : vocab // 3] -= 6
    elif kind == "zeros and just below":   # many of both: the bin below zero is counted again, beside zeros that are not in it
        x = torch.where(torch.rand(x.shape, generator=g) < 0.4, 0.0, -x.abs() * 1e-5)
        x[:, ::7] = -0.0
    elif kind == "zeros and around":
        x = torch.where(torch.rand(x.shape, generator=g) < 0.4, 0.0, x * 1e-4)
        x[:, 5] = 0.5
    elif kind == "negative":
        x = x - 40
    elif kind == "below the lowest bin":
        x = x * 30 - 500
    elif kind == "above the highest bin":
        x = x * 30 + 500
    elif kind == "both sides":
        x = x * 100
    elif kind == "lowest value":    # a mask of the type's lowest value
        x[torch.rand(x.shape, generator=g) < 0.9] = torch.finfo(dtype).min
    elif kind == "all lowest":
        x[:] = torch.finfo(dtype).min
    elif kind == "masked":
        x[torch.rand(x.shape, generator=g) < 0.99] = -math.inf
        x[:, 3] = 0.5
    elif kind == "one left":
        x[:] = -math.inf
        x[:, vocab - 1] = -3.0
    elif kind == "none left":
        x[:] = -math.inf
        x[0] = math.nan
    elif kind == "nan":
        x[torch.rand(x.shape, generator=g) < 0.2] = math.nan
        x[:, 0] = -math.nan
    elif kind == "infinite":
        x[:, 5::17] = math.inf
    elif kind == "infinite, one":
        x[:, 1] = math.inf
    return x.to(dtype)


KINDS = ["equal", "zeros", "two values", "tiny", "tiny, one ahead", "padded", "padded with both zeros", "zeros and just below", "zeros and around", "negative", "below the lowest bin", "above the highest bin", "both sides",
         "lowest value", "all lowest", "masked", "one left", "none left", "nan", "infinite", "infinite, one"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(2, 9001), (200, 700)])
def test_values(nv, kind, dtype, rows, vocab):
    x = special(kind, rows, vocab, dtype, 11)
    for i, kw in enumerate(({}, dict(k=7), dict(p=0.6), dict(m=0.5), dict(t=0.002), dict(t=30.0, p=0.5), dict(t=0.0), dict(t=math.inf, k=300))):
        check(nv, x, uniform(rows, i), **kw)


@pytest.mark.parametrize("dtype", TYPES)
def test_ends_of_the_random_numbers_and_of_the_settings(nv, dtype):
    u = torch.tensor([0.0, 2.0 ** -149, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan])
    n = len(u)
    x = logits(1, 2000, dtype, 2).expand(n, -1).contiguous()
    for kw in ({}, dict(k=3), dict(p=0.5), dict(m=0.1), dict(k=1), dict(k=2000), dict(k=1999), dict(k=-4), dict(p=0.0), dict(p=-1.0), dict(p=1.5),
               dict(p=math.nan), dict(m=1.0), dict(m=3.0), dict(m=-1.0), dict(m=math.nan), dict(t=-1.0), dict(t=math.nan), dict(k=2 ** 31 - 1)):
        check(nv, x, u, **kw)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_draws_from_one_row(nv, dtype):
    """Rows that are one row of memory (stride 0)."""
    x = logits(1, 5000, dtype, 8)
    many = x.cuda().expand(70, -1)
    check(nv, x.expand(70, -1), uniform(70, 3), p=0.9, device_x=many)
    check(nv, x.expand(70, -1), uniform(70, 4), t=0.5, device_x=many)


def test_a_whole_number_that_32_bits_do_not_hold(nv):
    x, u = logits(3, 900, torch.bfloat16, 2), uniform(3, 9)
    for k in (1 << 31, (1 << 32) + 3, -(1 << 40)):
        ids, _ = nv.sample(x.cuda(), u.cuda(), 1.0, k)
        assert torch.equal(ids, nv.sample(x.cuda(), u.cuda())[0])


def test_equal_tokens_are_drawn_by_index(nv):
    x = torch.zeros(8, 8, dtype=torch.bfloat16)
    u = torch.arange(8) / 8          # each exactly at a border: the token behind it
    assert check(nv, x, u).tolist() == list(range(8))
    assert check(nv, x, u, k=4).tolist() == [0, 0, 1, 1, 2, 2, 3, 3]
    assert check(nv, x, u, p=0.5).tolist() == [0, 0, 1, 1, 2, 2, 3, 3]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,stride,offset", [(1000, 1000, 0), (1001, 1001, 0), (777, 1003, 1), (777, 780, 3), (5, 9, 7), (20001, 20011, 5)])
def test_rows_at_odd_places(nv, dtype, vocab, stride, offset):
    """Rows that start anywhere; what lies between them is large and never drawn."""
    rows = 6
    x = logits(rows, vocab, dtype, vocab)
    flat = torch.full((offset + rows * stride + 16,), 90.0, dtype=dtype, device="cuda")
    view = flat[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    view.copy_(x)
    check(nv, x, uniform(rows, 1), device_x=view)
    check(nv, x, uniform(rows, 2), t=0.0, device_x=view)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3000, 70001])
def test_a_row_s_token_does_not_depend_on_the_batch(nv, dtype, vocab):
    """One row, a few, many: other numbers of CTAs take a row."""
    x, u = logits(400, vocab, dtype, 4).cuda(), uniform(400, 4).cuda()
    all_ids, all_probs = nv.sample(x, u, 0.9, 0, 0.95, 0.01)
    for n in (1, 7, 30, 100):
        ids, probs = nv.sample(x[:n], u[:n], 0.9, 0, 0.95, 0.01)
        assert torch.equal(ids, all_ids[:n]) and torch.equal(probs, all_probs[:n])


def test_draws_follow_the_probabilities(nv):
    """Evenly spaced random numbers: each token's share is its probability to one part in their number."""
    x = logits(1, 50, torch.bfloat16, 9, sigma=1.0)
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    ids, _ = nv.sample(x.expand(n, -1).contiguous().cuda(), u.cuda())
    share = torch.bincount(ids.cpu().long(), minlength=50).double() / n
    assert float((share - torch.softmax(x[0].double(), 0)).abs().max()) <= 1.0 / n + 1e-12


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,drafts,vocab", [(1, 0, 500), (3, 1, 1000), (8, 3, 4099), (5, 7, 300), (200, 2, 130)])
def test_verification(nv, dtype, batch, drafts, vocab):
    rows = batch * (drafts + 1)
    x, u = logits(rows, vocab, dtype, 6), uniform(rows, 6)
    g = torch.Generator().manual_seed(3)
    t, p = 0.5 + torch.rand(batch, generator=g), 0.7 + 0.3 * torch.rand(batch, generator=g)
    k = torch.randint(0, 40, (batch,), generator=g).int()
    each = lambda v: v.repeat_interleave(drafts + 1)
    want = check(nv, x, u, each(t), each(k), each(p)).view(batch, drafts + 1)
    # drafts that are right up to a place of their own
    right = torch.randint(0, drafts + 1, (batch,), generator=g)
    d = want[:, :drafts].clone()
    for b in range(batch):
        if right[b] < drafts:
            d[b, right[b]] = (d[b, right[b]] + 1) % vocab
    tokens, accepted, probs = nv.verify_sample(x.cuda(), u.cuda(), d.cuda(), t.cuda(), k.cuda(), p.cuda())
    assert torch.equal(tokens.cpu(), want) and torch.equal(accepted.cpu().long(), right)
    ids, q = nv.sample(x.cuda(), u.cuda(), each(t).cuda(), each(k).cuda(), each(p).cuda())
    assert torch.equal(ids.view_as(tokens), tokens) and torch.equal(q.view_as(probs), probs)


def test_refusals(nv):
    x, u = logits(4, 100, torch.bfloat16, 1).cuda(), uniform(4, 1).cuda()
    one = torch.ones(4, device="cuda")
    for args in ((x, u.double()), (x, u[:3]), (x, u.repeat(2)[::2]), (x, u, one.double()), (x, u, one[:3]), (x, u, 1.0, one), (x, u, 1.0, 0, one.view(2, 2)),
                 (x, u, 1.0, 0, 1.0, one.repeat(2)[::2])):
        with pytest.raises(ValueError):
            nv.sample(*args)
    for args in ((x, u.cpu()), (x, u, one.cpu()), (x, u, 1.0, one.int().cpu())):
        with pytest.raises(RuntimeError, match="CUDA"):
            nv.sample(*args)
    drafts = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for args in ((x, u, drafts.long()), (x, u, drafts[:1]), (x, u, drafts, one)):
        with pytest.raises(ValueError):
            nv.verify_sample(*args)
    with pytest.raises(RuntimeError, match="CUDA"):
        nv.verify_sample(x, u, drafts.cpu())
    with pytest.raises(RuntimeError, match="unsupported shape"):
        nv.sample(torch.zeros(1, 524289, dtype=torch.bfloat16, device="cuda"), u[:1])
    with pytest.raises(RuntimeError, match="invalid argument"):
        nv.sample(x[:, :0], u)
    ids, probs = nv.sample(x[:0], u[:0])
    assert ids.shape == probs.shape == (0,)
    tokens, accepted, probs = nv.verify_sample(x[:0], u[:0], drafts[:0])
    assert tokens.shape == probs.shape == (0, 2) and accepted.shape == (0,)


def test_in_a_graph_and_on_two_streams(nv):
    rows, vocab = 9, 20000
    x, u, t = logits(rows, vocab, torch.bfloat16, 1).cuda(), uniform(rows, 1).cuda(), torch.ones(rows, device="cuda")
    sides = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            nv.sample(x, u, t, 0, 0.9)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = nv.sample(x, u, t, 0, 0.9)
            graphs.append((g, out))
    torch.cuda.synchronize()
    for seed in (2, 3):
        nx, nu = logits(rows, vocab, torch.bfloat16, seed), uniform(rows, seed)
        x.copy_(nx)
        u.copy_(nu)
        torch.cuda.synchronize()
        for s, (g, _) in zip(sides, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = check(nv, nx, nu, p=0.9)
        for _, (ids, _) in graphs:
            assert torch.equal(ids.cpu(), want)


def test_behind_the_head(nv):
    """hidden -> norm -> W4A16 head -> draw, as one captured step feeds the next."""
    K, V, rows = 512, 3000, 4
    g = torch.Generator().manual_seed(5)
    head = nv.quantize(torch.randn(V, K, generator=g).cuda() * 0.1)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    h = torch.randn(rows, K, generator=g).bfloat16().cuda()
    u = uniform(rows, 5)
    y = nv.rms_norm(h, w)
    x = nv.gemm_w4a16(y, head)
    check(nv, x.cpu(), u, t=0.8, p=0.9, device_x=x)
