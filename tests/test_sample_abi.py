"""CPU-side checks of the draw's C ABI and Python calls: every refusal comes back before anything is launched."""
import pytest
import torch

from tests.test_abi import nv  # noqa: F401  (the built library)

P = 0x100000   # an aligned address that is never read


def one(m, logits=P, dtype=1, rows=4, vocab=100, stride=100, u=P, ids=P, probs=P):
    return m.lib().nvfp4_sample(logits, dtype, rows, vocab, stride, m.CSampling(None, None, None, None, 1.0, 0, 1.0, 0.0), u, ids, probs, None)


def verify(m, logits=P, dtype=1, batch=2, drafts=3, vocab=100, stride=100, u=P, draft_ids=P, ids=P, probs=P, acc=P):
    return m.lib().nvfp4_verify_sample(logits, dtype, batch, drafts, vocab, stride, m.CSampling(None, None, None, None, 1.0, 0, 1.0, 0.0), u, draft_ids, ids,
                                       probs, acc, None)


BAD = [(dict(logits=None), -1), (dict(u=None), -1), (dict(ids=None), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(vocab=0), -1), (dict(vocab=-5), -1),
       (dict(stride=99), -1), (dict(stride=-100), -1), (dict(stride=1), -1), (dict(vocab=524289, stride=1 << 20), -2), (dict(logits=P + 1), -3), (dict(logits=P + 2, dtype=0), -3)]


@pytest.mark.parametrize("kw,code", BAD)
def test_bad_logits(nv, kw, code):  # noqa: F811
    assert one(nv, **kw) == code
    assert verify(nv, **kw) == code


def test_rows(nv):  # noqa: F811
    assert one(nv, rows=-1) == -1 and one(nv, rows=(1 << 20) + 1) == -2
    assert one(nv, rows=0, logits=None, u=None, ids=None, probs=None) == 0
    assert verify(nv, batch=-1) == -1 and verify(nv, drafts=-1) == -1 and verify(nv, drafts=1 << 20) == -1
    assert verify(nv, batch=1 << 18, drafts=7) == -2
    assert verify(nv, draft_ids=None) == -1 and verify(nv, acc=None) == -1
    assert verify(nv, batch=0, logits=None, u=None, draft_ids=None, ids=None, probs=None, acc=None) == 0


def test_python_refusals(nv):  # noqa: F811
    x, u = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4)
    with pytest.raises(RuntimeError, match="CUDA"):
        nv.sample(x, u)
    for bad in (x.half(), x[0], x.double(), x.t()):
        with pytest.raises(ValueError, match="logits"):
            nv.sample(bad, u)
    with pytest.raises(ValueError, match="draft_ids"):
        nv.verify_sample(x, u, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows"):
        nv.verify_sample(x, u, torch.zeros(2, 2, dtype=torch.int32))
