"""The token-step example: norms, linears, attention and the draw together, captured and not."""
import pytest
import torch

from examples.token_step import Decoder, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("settings", [dict(), dict(temperature=0.0), dict(top_k=0, top_p=1.0, min_p=0.0, temperature=1.3)])
def test_captured_steps_draw_the_tokens_of_plain_calls(settings):
    a, pa = run(steps=12, graph=True, **settings)
    b, pb = run(steps=12, graph=False, **settings)
    assert torch.equal(a, b) and torch.equal(pa, pb)
    assert int(a.min()) >= 0 and int(a.max()) < Decoder.vocab
    assert bool((pa > 0).all() and (pa <= 1).all())
    if settings.get("temperature") == 0.0:
        assert bool((pa == 1).all())


def test_other_random_numbers_draw_other_tokens_only_where_there_is_a_choice():
    greedy, _ = run(steps=6, temperature=0.0)
    one, p = run(steps=6, top_k=1)
    assert torch.equal(greedy, one) and bool((p == 1).all())
    free, _ = run(steps=6, temperature=2.0, top_k=0, top_p=1.0, min_p=0.0)
    assert not torch.equal(greedy, free)
