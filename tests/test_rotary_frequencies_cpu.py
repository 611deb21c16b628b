"""The stretched frequencies' promise for every pair: those that make at least turns[0] turns over the
original context are kept, those that make at most turns[1] are divided by the factor."""
import math

import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb


@pytest.mark.parametrize("R", [2, 32, 128])
@pytest.mark.parametrize("length", [1, 6, 7, 40, 300, 4096, 1 << 20])
@pytest.mark.parametrize("turns", [(32.0, 1.0), (4.0, 2.0)])
def test_yarn_keeps_fast_pairs_and_divides_slow_ones(R, length, turns):
    f, _ = rb.rotary_frequencies(R)
    y, _ = rb.rotary_frequencies(R, scaling="yarn", factor=4.0, original_length=length,
                                 turns=turns)
    made = length * f / (2 * math.pi)
    fast, slow = made >= turns[0] * (1 + 1e-9), made <= turns[1] * (1 - 1e-9)
    assert torch.equal(y[fast], f[fast])
    assert torch.allclose(y[slow], f[slow] / 4, rtol=1e-12, atol=0)
    ratio = y / f
    assert bool((ratio[1:] <= ratio[:-1] + 1e-15).all()) and bool((ratio >= 0.25 - 1e-15).all())
