"""The sequence operators' refusals that are made on the host, without a GPU: through the C
entries, with addresses that nothing looks behind."""
import ctypes

import pytest
import torch

INVALID = 1


def _lib():
    from sparse_graph_recurrent_gb300 import _ck
    return _ck.load()


def reorder(states, parents, B, K, beams):
    """The status of ck_reorder_states for states (in, out, bytes, in_row, in_beam, out_row, out_beam)."""
    from sparse_graph_recurrent_gb300 import _ck
    array = (_ck.BeamState * len(states))(*(_ck.BeamState(*s) for s in states))
    return _lib().ck_reorder_states(array, len(states), ctypes.c_void_p(parents), B, K, beams, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused must find no device")
def test_parents_are_not_written():
    """An output over the parents would change them while others read them."""
    A, P = 1 << 40, 1 << 44
    size = 3 * 4 * 8
    assert reorder([(A, A + (1 << 30), 8, 32, 8, 32, 8)], P, 3, 4, 4) not in (0, INVALID)
    for at in (P, P + 8, P + size - 8, P - size + 8, P - 8):  # into new tensors, in part or whole
        assert reorder([(A, at, 8, 32, 8, 32, 8)], P, 3, 4, 4) == INVALID
    assert reorder([(P, P, 8, 32, 8, 32, 8)], P, 3, 4, 4) == INVALID  # in their own place
    for at in (P + size, P - size):  # beside them
        assert reorder([(A, at, 8, 32, 8, 32, 8)], P, 3, 4, 4) not in (0, INVALID)
    assert reorder([(P, A, 8, 32, 8, 32, 8)], P, 3, 4, 4) not in (0, INVALID)  # read as a state
