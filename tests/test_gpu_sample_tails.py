"""Draws from the tail of a peaked row: many light tokens whose masses have few bits each. bf16 and fp32 logits of the
same values name the same token, the one of the masses in whole numbers."""
import numpy as np
import pytest
import torch

from tests.gpu_common import nv as _nv
from tests.sample_masses import Row, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return _nv()


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return build(tmp_path_factory.mktemp("masses"))


def tail_numbers(row, n, seed):
    """Random numbers that fall into the row's tail, its first and last ones, and its end."""
    W, first = int(row.upto[-1]), int(row.upto[0])
    g = np.random.default_rng(seed)
    u = (first + g.random(n) * (W - first)) / W
    u = np.minimum(u.astype(np.float32), np.float32(1 - 2.0 ** -24))
    return np.concatenate((u, np.float32([0.0, first / W, 1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -22, 1.0, 2.0])))


def check(nv, lib, x, t, u, **kw):
    row = Row(lib, x.float().numpy(), t)
    want = [row.draw(float(v), **kw)[0] for v in u]
    uc = torch.from_numpy(u).cuda()
    n = len(u)
    for dtype in (torch.bfloat16, torch.float32):
        assert torch.equal(x.to(dtype).float(), x.float())
        one = x.to(dtype).cuda()
        ids, _ = nv.sample(one.expand(n, -1), uc, t, kw.get("k", 0), kw.get("p", 1.0), kw.get("m", 0.0))   # one CTA or a few for a row
        assert ids.tolist() == want, (dtype, [(i, a, b) for i, (a, b) in enumerate(zip(ids.tolist(), want)) if a != b][:3])
        for i in (n - 1, n - 2, n - 5, 0):                                                                # and many
            ids, _ = nv.sample(one[None], uc[i:i + 1], t, kw.get("k", 0), kw.get("p", 1.0), kw.get("m", 0.0))
            assert int(ids[0]) == want[i], (dtype, i)


@pytest.mark.parametrize("best", [12.0, 18.0, 20.0, 23.0, 25.0, 27.0])
@pytest.mark.parametrize("zeros", [50000, 200000])
def test_one_logit_above_a_padded_vocabulary(nv, lib, best, zeros):
    x = torch.zeros(zeros + 1)
    x[zeros // 3] = best
    x[5::3] = -0.0
    u = tail_numbers(Row(lib, x.numpy(), 1.0), 40, int(best))
    for kw in ({}, dict(p=1 - 2.0 ** -24), dict(p=0.9999), dict(k=zeros // 2), dict(m=1e-11), dict(k=zeros, p=1 - 2.0 ** -23)):
        check(nv, lib, x, 1.0, u, **kw)


@pytest.mark.parametrize("best,t", [(16.0, 1.0), (27.0, 1.0), (40.0, 1.5), (6.0, 0.25), (0.01, 0.0004), (0.02, 1.0)])
@pytest.mark.parametrize("vocab,tiny", [(3001, 400), (100000, 400), (100000, 20000)])
def test_one_logit_above_values_next_to_zero(nv, lib, best, t, vocab, tiny):
    """The bins on either side of zero, with as many values as are noted and with more; lists and finer counts of them."""
    g = torch.Generator().manual_seed(vocab + tiny)
    x = torch.full((vocab,), -30.0)
    at = torch.randperm(vocab, generator=g)[:tiny]
    x[at] = (torch.randn(tiny, generator=g) * 2e-4).clamp(-9e-4, 9e-4)
    x[at[::5]] = 0.0
    x[at[1::5]] = -0.0
    x[vocab // 2] = best
    x = x.bfloat16().float()
    u = tail_numbers(Row(lib, x.numpy(), t), 40, vocab)
    for kw in ({}, dict(p=0.99999), dict(k=tiny // 2), dict(m=1e-10)):
        check(nv, lib, x, t, u, **kw)


@pytest.mark.parametrize("depth", [10.0, 23.0, 29.0, 31.25])
def test_flat_tails(nv, lib, depth):
    """Two tokens next to each other above a flat tail, down to weights that are rounded away."""
    x = torch.full((248320,), -depth)
    x[0], x[1] = 0.0, -2.0 ** -29
    u = tail_numbers(Row(lib, x.numpy(), 1.0), 30, 1)
    u = np.concatenate((u, np.float32([0.5, 0.25, 0.75])))
    for kw in ({}, dict(p=0.999999), dict(m=2e-13), dict(k=100000)):
        check(nv, lib, x, 1.0, u, **kw)


@pytest.mark.parametrize("t", [3e38, 1e38, 2e37, 2.0 ** 64, 2.0 ** 63.5, 2.0 ** -63.9, 2.0 ** -64.1, 1e-37, 2.0 ** -128, 2.0 ** -149])
def test_temperatures_at_the_ends_of_fp32(nv, lib, t):
    """Logits as far apart as such a temperature asks for; next to the largest number their difference overflows."""
    t = float(np.float32(t))
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5000, generator=g).double() * 3 * t
    x = x.clamp(-3e38, 3e38).float().bfloat16().float()
    x[7], x[8] = max(float(x.max()), min(9 * t, 3e38)), -3e38
    x = x.bfloat16().float()
    u = np.concatenate((np.random.default_rng(1).random(40).astype(np.float32), np.float32([0.0, 0.5, 1 - 2.0 ** -24, 1.0])))
    for kw in ({}, dict(p=0.7), dict(k=40), dict(m=0.01)):
        check(nv, lib, x, t, u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_logits_whose_difference_overflows(nv, dtype):
    """3 10^38 and its negative at a temperature of 3 10^38: the second token weighs e^-2."""
    x = torch.tensor([[3e38, -3e38]]).to(dtype)
    t = float(np.float32(3e38))
    u = torch.tensor([0.0, 0.5, 0.87, 0.89, 0.95])
    ids, probs = nv.sample(x.cuda().expand(5, -1), u.cuda(), t)
    share = 1 / (1 + np.exp(-2 * float(x[0, 0].double()) / t))
    assert ids.tolist() == [int(float(v) > share) for v in u] == [0, 0, 0, 1, 1]
    want = torch.tensor([share, share, share, 1 - share, 1 - share])
    assert bool(((probs.cpu().double() - want).abs() <= 2.0 ** -22).all())
