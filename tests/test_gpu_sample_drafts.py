"""Verification by sampling where positions have no token: a -1 is none, so a draft of -1 (a padded list) never stands."""
import math

import pytest
import torch

from tests.gpu_common import nv as _nv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [0.0, 1.0])
def test_a_position_without_a_token_accepts_nothing(dtype, t):
    nv = _nv()
    batch, drafts, vocab = 3, 2, 300
    g = torch.Generator().manual_seed(1)
    x = torch.randn(batch, drafts + 1, vocab, generator=g)
    x[0] = -math.inf           # no token anywhere
    x[1, 1] = math.nan         # none behind the first draft
    x = x.view(-1, vocab).to(dtype)
    u = torch.rand(batch * (drafts + 1), generator=g)
    ids, _ = nv.sample(x.cuda(), u.cuda(), t)
    want = ids.view(batch, drafts + 1).cpu()
    assert want[0].tolist() == [-1, -1, -1] and int(want[1, 1]) == -1 and int(want[1, 0]) >= 0
    d = want[:, :drafts].clone()
    tokens, accepted, probs = nv.verify_sample(x.cuda(), u.cuda(), d.cuda(), t)
    assert torch.equal(tokens.cpu(), want)
    assert accepted.tolist() == [0, 1, 2]
    assert not probs[0].any() and float(probs[1, 1]) == 0
    # padded lists in ordinary rows
    d[2, 1] = -1
    assert nv.verify_sample(x.cuda(), u.cuda(), d.cuda(), t)[1].tolist() == [0, 1, 1]
