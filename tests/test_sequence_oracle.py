"""The definitions of sequence_oracle.py against differences and closed forms, on the CPU."""
import numpy as np
import pytest

import sequence_oracle as so


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("lengths", [None, (5, 0)])
def test_gradients_of_the_gated_recurrence_are_differences(form, lengths):
    rng = np.random.default_rng(3)
    T, B, N = 6, 2, 3
    x, gate, h0 = rng.normal(size=(T, B, N)), rng.normal(size=(T, B, N)), rng.normal(size=(B, N))
    d, ds = rng.normal(size=(T, B, N)), rng.normal(size=(B, N))
    lengths = None if lengths is None else np.array(lengths)
    got, _ = so.gated(x, gate, h0, lengths, form, d, ds)

    def loss(x, gate, h0):
        v, _ = so.gated(x, gate, h0, lengths, form)
        return (v["out"] * d).sum() + (v["state"] * ds).sum()

    args, e = [x, gate, h0], 1e-5
    for k, name in enumerate(("dx", "dgate", "dstate0")):
        want = np.zeros_like(args[k])
        for i in np.ndindex(want.shape):
            at = [a.copy() for a in args]
            at[k][i] += e
            up = loss(*at)
            at[k][i] -= 2 * e
            want[i] = (up - loss(*at)) / (2 * e)
        # third derivatives of a few units times e^2 / 6, and 1e-16 / e
        assert np.abs(got[name] - want).max() < 1e-8, name


def test_a_constant_decay_is_a_geometric_sum():
    T = 9
    got, _ = so.gated(np.ones((T, 1, 1)), np.full((T, 1, 1), 0.5), None, None, "decay")
    assert np.allclose(got["out"][:, 0, 0], 2 - 0.5 ** np.arange(T))


def test_beams_of_a_small_case_by_hand():
    z = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]]]))
    s, p, t, e = so.beam(z, np.log(np.array([[0.5, 0.5]])), None, 2, 3)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[2, 0, 1]] and e.tolist() == [[True, False, False]]
    assert np.allclose(np.exp(s), [[0.35, 0.25, 0.125]])


def test_clipping_by_hand():
    norm, factor = so.clip([np.array([3.0]), np.array([4.0])], 2.5)
    assert norm == 5 and abs(factor - 0.5) < 1e-6 and so.clip([np.array([3.0])], 4)[1] == 1
