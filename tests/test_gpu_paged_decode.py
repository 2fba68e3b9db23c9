"""The serving loop of examples/paged_decode.py: decoding token by token in a
captured graph, over forked and compacted pages, agrees with reading the whole
sequences in one chunk."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_steps_agree_with_one_chunk(kv):
    import paged_decode
    stepwise, at_once = paged_decode.run(kv, steps=20)
    # both sides round q, k, v, the attention output and the block's output to
    # bf16 (2^-9 each) from sums taken in another order, and the chunk rounds its
    # weights p to bf16 or f16: a few times 2^-9
    err = ((stepwise.float() - at_once.float()).norm() / at_once.float().norm()).item()
    assert err <= 1e-2, err
