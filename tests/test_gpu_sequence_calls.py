"""Calls of the sequence operators that their documentation allows at its borders: one step of a
wider array, outputs laid out otherwise than the gradients, lists with nothing in them, views
that are conjugated or negated lazily, as many beams and tokens as there may be."""
import numpy as np
import pytest
import torch

import sequence_oracle as so
from test_gpu_clip import FACTOR_OFF, NORM_OFF
from test_gpu_gated import TYPES, check, inputs

pytestmark = pytest.mark.gpu


def host(t):
    return t.detach().double().cpu().numpy()


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
# -- clipping --------------------------------------------------------------------------------


def clipped(grads, out, max_norm):
    """Clips grads into out and looks at all that may and may not change."""
    import sparse_graph_recurrent_gb300 as ck
    want = [host(g) for g in grads]
    before = [(g, g.clone(), g._version) for g in grads]
    norm, factor = so.clip(want, max_norm)
    got = ck.clip_gradients(grads, max_norm, out=out)
    assert abs(float(got) - norm) <= NORM_OFF * norm
    for o, w in zip(out, want):
        so.within(host(o), w * factor, np.abs(w * factor) * FACTOR_OFF, str(o.dtype)[6:])
    assert all(torch.equal(g, was) and g._version == version for g, was, version in before)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_gradients_stay_as_they_are_wherever_out_lies(max_norm, dtype):
    dt = TYPES[dtype]
    new = lambda *n: torch.randn(*n, device="cuda").to(dt)  # noqa: E731
    zeros = lambda *n: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    for lay in (lambda: zeros(4, 12)[:, ::2], lambda: zeros(6, 4).t(), lambda: zeros(4, 9)[:, 2:8], lambda: zeros(8, 6)[::2],
                lambda: zeros(4, 6)):
        for grad in (lambda: new(4, 6), lambda: new(6, 4).t(), lambda: new(4, 12)[:, 1::2]):
            clipped([grad()], [lay()], max_norm)
            clipped([new(7), grad(), new(4, 6)], [zeros(7), lay(), zeros(12, 4).t()[:, 3:9]], max_norm)
    wide = torch.full((50, 90), 7.0, dtype=dt, device="cuda")
    clipped([new(50, 40)], [wide[:, 20:60]], max_norm)  # what lies beside is as it was
    assert (wide[:, :20] == 7).all() and (wide[:, 60:] == 7).all()
    lines = zeros(2, 3000)
    clipped([new(3000)], [lines.t()[:, 1]], max_norm)
    assert not lines[0].any()


@pytest.mark.parametrize("count", [1000, 2000, 1001])
@pytest.mark.parametrize("empty", [1, 3])
def test_empty_tensors_behind_a_full_list(count, empty):
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator().manual_seed(count)
    for apart in (False, True):
        grads = [torch.randn(1 + i % 50, generator=g).cuda() for i in range(count)]
        grads[5:5] = [torch.empty(0, device="cuda")] * (count % 1000)  # (more than a launch's, and some in between)
        grads += [torch.empty(0, device="cuda") for _ in range(empty)]
        out = [torch.full_like(t, 9) for t in grads] if apart else grads
        want = [host(t) for t in grads]
        norm, factor = so.clip(want, 0.5)
        got = ck.clip_gradients(grads, 0.5, out=out if apart else None)
        assert abs(float(got) - norm) <= NORM_OFF * norm and factor < 1
        for t, w in zip(out, want):
            so.within(host(t), w * factor, np.abs(w * factor) * FACTOR_OFF)
        assert abs(float(ck.grad_norm(out)) - 0.5) < 1e-5
