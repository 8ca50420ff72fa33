"""The example that trains a feed-forward block and decodes with packed weights.

Decoding differs from the trained block by the rounding of the down projection
to four bits: a group's scale s is below amax / 3, a weight below 2 s moves by at
most s / 4 and one above by a fifth of itself.  Of 32 weights of a normal
distribution amax is some 2.1 deviations, which puts the root mean square of the
rounding near 0.15 of the weights' own; a third is allowed.
"""

import numpy as np
import pytest
import torch

from examples import feed_forward

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_decode_agrees():
    losses, norms, one_by_one, together = feed_forward.run(features=256, hidden=384, tokens=200, steps=12)
    assert np.all(np.isfinite(losses)) and np.all(np.isfinite(norms)) and min(norms) > 0
    assert losses[-1] < losses[0]
    a, b = one_by_one.double(), together.double()
    assert a.shape == b.shape == (4, 256) and float((a - b).norm()) < float(b.norm()) / 3


def test_decode_is_repeatable_and_takes_any_rows():
    torch.manual_seed(1)
    decode = feed_forward.Decoder(feed_forward.FeedForward(256, 384, None, "cuda:0"))
    x = torch.randn(5, 256, device="cuda:0").bfloat16()
    assert torch.equal(decode(x), decode(x))
    h = [decode(x[i:i + 1]) for i in range(5)]
    assert all(t.shape == (1, 256) and torch.isfinite(t).all() for t in h)
