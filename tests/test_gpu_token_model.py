"""The readout operators together, as examples/token_model.py runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_example_learns_and_answers():
    import token_model as tm
    losses, got = tm.main(["--steps", "120", "--tokens", "20", "--nodes", "256"])
    # ln 256 = 5.5 before training; the text's bytes are nearly always told by those before
    assert losses[0] > 4.0 and losses[-1] < 0.5 * losses[0]
    assert got.shape == (2, 20)
    assert all(b in tm.TEXT for row in got.tolist() for b in row)  # the mask's bytes only


def test_answers_repeat_and_follow_the_seed():
    import token_model as tm
    torch.manual_seed(0)
    model = tm.Model(128, 1024, 16, torch.device("cuda"))
    p = [tm.TEXT[:8]] * 3
    a, b, c = (tm.answer(model, p, 12, seed=s, temperature=1.5) for s in (1, 1, 2))
    assert torch.equal(a, b) and not torch.equal(a, c)
    assert not torch.equal(a[0], a[1])  # rows of one batch draw apart
