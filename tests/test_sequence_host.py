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


def meet(a, b):
    """Whether two arrays (lo, row, beam, rows, beams, bytes) share a byte, from all of theirs."""
    def every(e):
        lo, row, beam, rows, beams, n = e
        return {lo + i * row + j * beam + k for i in range(rows) for j in range(beams) for k in range(n)}
    return bool(every(a) & every(b))


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused must find no device")
def test_what_is_taken_for_sharing_memory():
    """Nothing that shares a byte is let through; halves and columns of one array, in any order of
    its axes, are."""
    import random
    A = 1 << 40
    rng = random.Random(5)
    known = 0
    for i in range(4000):
        B, K, n = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 6)
        row, beam = rng.choice([(K * n, n), (2 * K * n, n), (K * n * 2, 2 * n), (n, B * n), (n, 2 * B * n), (2 * n, 2 * B * n),
                                (rng.randint(1, 60), rng.randint(1, 60))])
        orow, obeam = rng.choice([(row, beam), (row, beam), (2 * row, beam), (rng.randint(1, 60), rng.randint(1, 60))])
        at = rng.choice([0, n, K * n, B * n, B * K * n, rng.randint(-40, 40), -K * n, -n])
        if at == 0:
            continue
        got = reorder([(A, A + at, n, row, beam, orow, obeam)], 1 << 44, B, K, K)
        own = len({A + at + i * orow + j * obeam + k for i in range(B) for j in range(K) for k in range(n)}) < B * K * n
        shared = meet((A, row, beam, B, K, n), (A + at, orow, obeam, B, K, n))
        if own or shared:
            assert got == INVALID, (B, K, n, row, beam, orow, obeam, at)
        known += got != INVALID
    assert known > 1000
    N = 33 * 4
    for row, beam, at in ((8 * N, N, 4 * N), (4 * N, N, 12 * N), (8 * N, 2 * N, N), (N, 6 * N, 3 * N), (8 * N, N, -4 * N),
                          (N, 6 * N, -3 * N), (8 * N, 2 * N, -N)):
        assert not meet((0, row, beam, 3, 4, N), (at, row, beam, 3, 4, N))
        assert reorder([(A, A + at, N, row, beam, row, beam)], 1 << 44, 3, 4, 4) not in (0, INVALID)


def test_strided_tensors_that_may_share_memory():
    """What is taken to lie side by side does, whatever the strides; plain cases are."""
    import random

    from sparse_graph_recurrent_gb300.gradients import _Span
    rng = random.Random(2)
    line = torch.arange(4000, dtype=torch.float32)
    known = 0
    for _ in range(3000):
        views = []
        for _ in range(2):
            shape = [rng.randint(1, 5) for _ in range(rng.randint(1, 3))]
            stride = [rng.choice([1, 2, 3, 6, 12, 24, rng.randint(0, 40)]) for _ in shape]
            views.append(torch.as_strided(line, shape, stride, rng.randint(0, 60)))
        a, b = sorted(views, key=lambda t: t.data_ptr())
        shared = bool(set(a.flatten().tolist()) & set(b.flatten().tolist()))
        a, b = _Span(a, True), _Span(b, True)
        apart = b.lo >= a.hi or a.beside(b)
        assert not (shared and apart)
        known += apart and not shared
    assert known > 500


def test_what_clipping_takes_and_refuses_of_strided_tensors():
    """A tensor's own place is its own however it is named: the strides of axes of one do not count."""
    from sparse_graph_recurrent_gb300.gradients import _refuse_shared
    w, to = torch.zeros(8, 12), torch.zeros(8, 12)
    row = w[7:, :5]
    for pairs in ([(row, row)], [(row, row.as_strided((1, 5), (3, 1), row.storage_offset()))], [(w[:, ::2], w[:, ::2]), (w[:, 1::2], to)],
                  [(w[:, :0], w[:, :0]), (w, w)], [(w[:, 0], to[:, 3]), (w[:, 1], to[:, 2])]):
        _refuse_shared(pairs)
    for pairs in ([(row, row.as_strided((1, 5), (3, 2), row.storage_offset()))], [(w[:, ::2], w[:, 1::2]), (w[:, 1::2], to)],
                  [(w[:, :3], to[:, :1].expand(8, 3))], [(w[:, 0], to[:, 3]), (to[0], w[1])]):
        with pytest.raises(ValueError):
            _refuse_shared(pairs)
