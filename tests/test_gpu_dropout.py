"""Counter-based dropout against its definition in numpy.  For each element the
result is one 32-bit product, rounded once more to a 16-bit type, so the
comparison is exact; the gradient is the same map of the output's gradient."""
import numpy as np
import pytest
import torch

import readout_oracle as ro

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def expected(x, p, seed, step, locked):
    keep = torch.from_numpy(ro.keep_mask(tuple(x.shape), p, seed, step, locked).copy())
    scale = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    v = (x.cpu().float() * float(scale)).to(x.dtype)
    return torch.where(keep, v, torch.zeros((), dtype=x.dtype))


def same(a, b):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    assert torch.equal(torch.nan_to_num(a, 12345.0), torch.nan_to_num(b, 12345.0))


def data(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("locked", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (2, 1, 5), (3, 4, 8), (8, 8, 256), (5, 3, 1031),
                                   (7, 2, 3, 65), (2, 20, 4999), (33, 1, 4096), (3, 1, 70001)])
def test_matches_the_definition(shape, locked, dtype):
    import sparse_graph_recurrent_gb300 as ck
    x = data(shape, dtype, 3)
    same(ck.dropout(x, 0.3, 99, 5, locked=locked), expected(x, 0.3, 99, 5, locked))


@pytest.mark.parametrize("p", [0.0, 1e-12, 0.1, 0.5, 0.999, 1.0 - 1e-12, 1.0])
def test_probabilities(p):
    import sparse_graph_recurrent_gb300 as ck
    x = data((3, 1003), torch.float32)
    y = ck.dropout(x, p, 2 ** 63 + 11, 2 ** 40 + 3)
    same(y, expected(x, p, 2 ** 63 + 11, 2 ** 40 + 3, False))
    if p == 0.0:
        assert torch.equal(y, x)
    if p == 1.0:
        assert not y.any()


VIEWS = {
    "rows_cut": lambda b: b[:4 * 6 * 130].view(4, 6, 130)[..., :121],
    "rows_cut_odd_start": lambda b: b[3:3 + 4 * 6 * 130].view(4, 6, 130)[..., 1:122],
    "odd_pitch": lambda b: b[1:1 + 4 * 6 * 129].view(4, 6, 129)[..., :128],
    "odd_start": lambda b: b[1:1 + 2 * 4096].view(2, 1, 4096),
    "transposed": lambda b: b[:4 * 6 * 37].view(6, 4, 37).transpose(0, 1),
    "innermost_strided": lambda b: b[:4 * 6 * 64].view(4, 6, 64)[..., ::2],
    "innermost_swapped": lambda b: b[:4 * 6 * 40].view(4, 40, 6).transpose(1, 2),
    "expanded": lambda b: b[:45].view(1, 1, 45).expand(4, 6, 45),
    "scalar_expanded": lambda b: b[:1].view(1, 1, 1).expand(4, 6, 45),
    "four_axes": lambda b: b[:3 * 2 * 5 * 40].view(3, 2, 5, 40).permute(3, 0, 2, 1)[::2],
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("locked", [False, True])
@pytest.mark.parametrize("view", list(VIEWS))
def test_strides(view, locked, dtype):
    import sparse_graph_recurrent_gb300 as ck
    x = VIEWS[view](data((10000,), dtype, 8))
    y = ck.dropout(x, 0.4, 7, 1, locked=locked)
    assert y.is_contiguous()
    same(y, expected(x, 0.4, 7, 1, locked))


@pytest.mark.parametrize("cut", [0, 5])
def test_more_than_two_to_the_31_elements(cut):
    """Element indexes past 32 bits, dense and in rows cut out of wider ones: windows at
    both ends and around 2^31 and 2^32 are compared."""
    import sparse_graph_recurrent_gb300 as ck
    rows, n = 5, 900_000_000
    base = torch.ones(rows, n + cut, dtype=torch.bfloat16, device="cuda")
    y = ck.dropout(base[:, :n], 0.3, 17, 3).view(-1)
    for at in (0, n - 500, 2 ** 31 - 500, 2 ** 32 - 500, rows * n - 1000):
        w = ro.philox_words(np.arange(at, at + 1000), 17, 3)
        want = torch.from_numpy((w.astype(np.int64) >= int(np.rint(0.3 * 2 ** 32))))
        assert torch.equal(y[at:at + 1000].cpu() > 0, want), at


def test_dropped_values_are_zero_whatever_they_hold():
    import sparse_graph_recurrent_gb300 as ck
    x = data((4, 4099), torch.float32)
    x[0] = float("nan")
    x[1] = float("inf")
    x[2] = -3e38
    same(ck.dropout(x, 0.5, 5, 6), expected(x, 0.5, 5, 6, False))


def test_gradient_is_the_same_mask_and_matches_differences():
    import sparse_graph_recurrent_gb300 as ck
    x = data((6, 3, 77), torch.float32, 4).requires_grad_()
    d = data((6, 3, 77), torch.float32, 5)
    for locked in (False, True):
        y = ck.dropout(x, 0.25, 13, 21, locked=locked)
        (dx,) = torch.autograd.grad(y, x, d)
        same(dx, expected(d, 0.25, 13, 21, locked))
        same(ck.dropout_backward(d, 0.25, 13, 21, locked=locked), dx)
        # the map is linear, so a difference quotient is exact but for rounding: two products
        # of relative error 2^-24 each, over a step of 2
        with torch.no_grad():
            up, dn = (ck.dropout(x + e, 0.25, 13, 21, locked=locked).double() for e in (1.0, -1.0))
        quotient = (up - dn) / 2 * d.double()
        bound = 2.0 ** -22 * (x.detach().abs().double() + 1.0) * 2 * d.abs().double()
        assert ((quotient - dx.double()).abs() <= bound).all()


def test_gradient_of_a_sum_and_of_a_view():
    """An expanded output gradient (stride 0) and an input that is a view."""
    import sparse_graph_recurrent_gb300 as ck
    base = data((5, 64, 30), torch.float32).requires_grad_()
    y = ck.dropout(base.transpose(1, 2)[..., :50], 0.5, 3, 4, locked=True)
    y.sum().backward()
    want = torch.zeros(5, 64, 30)
    want[:, :50] = expected(torch.ones(5, 30, 50), 0.5, 3, 4, True).transpose(1, 2)
    same(base.grad, want)


def test_every_step_and_seed_is_a_stream_of_its_own():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.ones(1 << 20, device="cuda")
    a = ck.dropout(x, 0.5, 1, 1) > 0
    for seed, step in ((1, 2), (2, 1), (1 + 2 ** 32, 1), (1, 1 + 2 ** 32)):
        b = ck.dropout(x, 0.5, seed, step) > 0
        # agreeing elements are binomial(2^20, 1/2): 6 standard deviations are 3072
        assert abs(int((a == b).sum()) - (1 << 19)) < 3072
    assert abs(int(a.sum()) - (1 << 19)) < 3072


def test_step_on_the_device_and_capture():
    """A captured step draws anew on each replay, and the gradient keeps its forward's mask."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    x = data((9, 517), torch.float32)
    step = torch.tensor([7], dtype=torch.int64, device="cuda")
    same(ck.dropout(x, 0.3, 1, step), expected(x, 0.3, 1, 7, False))
    xr = x.clone().requires_grad_()
    y = ck.dropout(xr, 0.3, 1, step)
    _ck.ck_step_advance(step)  # before the backward
    y.backward(x)
    same(xr.grad, expected(x, 0.3, 1, 7, False))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ck.dropout(x, 0.3, 1, step)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ck.dropout(x, 0.3, 1, step)
        _ck.ck_step_advance(step)
    for k in (8, 9, 10):
        graph.replay()
        same(out, expected(x, 0.3, 1, k, False))


def test_side_stream_and_empty():
    import sparse_graph_recurrent_gb300 as ck
    x = data((64, 1000), torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = ck.dropout(x, 0.5, 1, 1)
    s.synchronize()
    same(y, expected(x, 0.5, 1, 1, False))
    for shape in ((0,), (0, 4), (4, 0), (3, 0, 5)):
        z = torch.empty(shape, device="cuda")
        assert ck.dropout(z, 0.5, 1).shape == shape
    assert ck.dropout(torch.ones((), device="cuda"), 0.0, 1).shape == ()


def test_refusals():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.ones(4, 4, device="cuda")
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ck.CKError) as e:
            ck.dropout(x, p, 1)
        assert e.value.name == "CK_ERR_INVALID_ARG"
    with pytest.raises(ValueError):
        ck.dropout(x.double(), 0.5, 1)
    with pytest.raises(ValueError):
        ck.dropout(x[0], 0.5, 1, locked=True)
    with pytest.raises(ValueError):
        ck.dropout(x, 0.5, 1, torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        ck.dropout(x, 0.5, 1, torch.tensor([1]))
    with pytest.raises(ValueError):
        ck.dropout(x, 0.5, 1, torch.tensor([1], dtype=torch.int32, device="cuda"))


def test_second_derivatives():
    """A penalty on the gradient through dropout: with y = m x^2 (m the factor or 0) and
    f = sum y^2, f' = 4 m^2 x^3 and sum f'^2 has the gradient 96 m^4 x^5."""
    import sparse_graph_recurrent_gb300 as ck
    for locked in (False, True):
        x = (data((3, 4, 65), torch.float32, 6) / 4).double().float().requires_grad_()
        y = ck.dropout(x * x, 0.25, 13, 21, locked=locked)
        (g,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
        assert g.requires_grad
        (h,) = torch.autograd.grad((g * g).sum(), x)
        m = torch.from_numpy(ro.keep_mask((3, 4, 65), 0.25, 13, 21, locked).copy()).double() / 0.75
        xd = x.detach().double().cpu()
        # a dozen roundings of 2^-24 each at most on either
        assert ((g.detach().double().cpu() - 4 * m ** 2 * xd ** 3).abs() <= 2.0 ** -20 * (4 * m ** 2 * xd ** 3).abs() + 1e-35).all()
        want = 96 * m ** 4 * xd ** 5
        assert ((h.double().cpu() - want).abs() <= 2.0 ** -18 * want.abs() + 1e-35).all()


def test_second_derivatives_keep_the_forwards_step():
    """The counter moves on between the forward, the gradient and the gradient's gradient."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    step = torch.tensor([7], dtype=torch.int64, device="cuda")
    x = data((5, 130), torch.float32, 1).requires_grad_()
    d = data((5, 130), torch.float32, 2).requires_grad_()
    y = ck.dropout(x, 0.5, 3, step)
    _ck.ck_step_advance(step)
    (g,) = torch.autograd.grad(y, x, d, create_graph=True)
    _ck.ck_step_advance(step)
    (h,) = torch.autograd.grad(g, d, torch.ones_like(g))
    same(g.detach(), expected(d.detach(), 0.5, 3, 7, False))
    same(h, expected(torch.ones(5, 130), 0.5, 3, 7, False))


def test_the_gradient_call_is_differentiable():
    import sparse_graph_recurrent_gb300 as ck
    d = data((4, 99), torch.float32, 2).requires_grad_()
    g = ck.dropout_backward(d, 0.3, 5, 6)
    (h,) = torch.autograd.grad(g, d, torch.ones_like(g))
    same(h, expected(torch.ones(4, 99), 0.3, 5, 6, False))
    with torch.no_grad():
        assert not ck.dropout_backward(d, 0.3, 5, 6).requires_grad


def test_forward_mode():
    """The tangent of dropout is dropout of the tangent, with the same mask; of a tangent
    that requires a gradient it stays differentiable."""
    import torch.autograd.forward_ad as fwd

    import sparse_graph_recurrent_gb300 as ck
    x, t = data((6, 3, 77), torch.float32, 4), data((6, 3, 77), torch.float32, 5)
    for locked in (False, True):
        for v in (x, x.transpose(1, 2)):
            with fwd.dual_level():
                for call in (ck.dropout, ck.dropout_backward):
                    y = fwd.unpack_dual(call(fwd.make_dual(v, t.view(v.shape)), 0.25, 13, 21, locked=locked))
                    same(y.primal, expected(v, 0.25, 13, 21, locked))
                    same(y.tangent, expected(t.view(v.shape), 0.25, 13, 21, locked))
    with fwd.dual_level(), torch.no_grad():
        assert fwd.unpack_dual(ck.dropout(fwd.make_dual(x, t), 0.25, 13)).tangent is not None
    leaf = t.clone().requires_grad_()
    with fwd.dual_level():
        y = fwd.unpack_dual(ck.dropout(fwd.make_dual(x, leaf), 0.25, 13, 21)).tangent
        (g,) = torch.autograd.grad(y, leaf, torch.ones_like(y))
    same(g, expected(torch.ones_like(x), 0.25, 13, 21, False))
    with fwd.dual_level():  # a level alone changes nothing
        same(ck.dropout(x, 0.25, 13, 21), expected(x, 0.25, 13, 21, False))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_locked_mask_past_two_to_the_34_elements(dtype):
    """A mask whose length is 4 mod 8, so that its repeats begin in the middle of 16 bytes,
    and long enough that the generator's block number carries into its high word."""
    import sparse_graph_recurrent_gb300 as ck
    n2, n3 = 1048321, 16388
    period = n2 * n3
    assert period > 2 ** 34 and period % 8 == 4
    if torch.cuda.mem_get_info()[0] < 2 * period * 2 + 2 ** 34:
        pytest.skip("needs 80 GB of device memory")
    row = torch.ones(n3, dtype=dtype, device="cuda")
    y = ck.dropout(row.expand(2, n2, n3), 0.5, 13, 3, locked=True).view(2, period)
    for at in (0, 2 ** 33 - 40, 2 ** 34 - 40, period - 80):
        w = ro.philox_words(np.arange(at, at + 80), 13, 3).astype(np.int64)
        want = torch.from_numpy(w >= 2 ** 31)
        for k in (0, 1):
            assert torch.equal(y[k, at:at + 80].cpu() > 0, want), (at, k)
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [8, 12, 10, 9, 2052])
def test_locked_masks_whose_repeats_begin_anywhere(n, dtype):
    """Periods of every remainder, dense and in rows cut out of wider ones."""
    import sparse_graph_recurrent_gb300 as ck
    for cut in (0, 3):
        x = data((5, 3, n + cut), dtype, n)[..., :n]
        same(ck.dropout(x, 0.4, 7, 2 ** 35 + 1, locked=True), expected(x, 0.4, 7, 2 ** 35 + 1, True))
