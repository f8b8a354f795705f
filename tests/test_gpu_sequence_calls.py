"""Calls of the sequence operators that their documentation allows at its borders: one step of a
wider array, outputs laid out otherwise than the gradients, lists with nothing in them, views
that are conjugated or negated lazily, as many beams and tokens as there may be."""
import numpy as np
import pytest
import torch

import sequence_oracle as so
from test_gpu_gated import TYPES, check, inputs

pytestmark = pytest.mark.gpu


# -- gated recurrence ------------------------------------------------------------------------


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [2, 6, 10, 14, 38, 70])
def test_one_step_of_a_wider_array(N, dtype, form):
    """[1, 1, N] taken from rows of any other length: the stride of its only step is odd, or no
    multiple of a pack, where rows are at multiples of packs but not of 16 bytes."""
    for width in (N + 7, N + 1, 2 * N + 1, N + 3, N + 2):
        for named in (("gate",), ("x",), ("x", "gate", "d_out"), ("d_out",)):
            d = inputs(1, 1, N, dtype, form, seed=N + width)
            for name in named:
                row = torch.full((1, width), float("nan"), dtype=TYPES[dtype], device="cuda")
                row[:, :N] = d[name][0]
                d[name] = row[:, :N][None]
                assert d[name].stride() == (width, width, 1)
            check(d, form, dtype)
