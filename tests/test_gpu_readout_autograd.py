"""What autograd is told by the readout operators that have no derivative."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_what_has_no_derivative_refuses_tangents():
    import torch.autograd.forward_ad as fwd

    import sparse_graph_recurrent_gb300 as ck
    w = torch.randn(40, 64, device="cuda")
    q, s, _ = ck.int4_quantize(w, 32)
    x = torch.randn(2, 64, device="cuda")
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: ck.int4_matvec(dual, q, s, group_size=32), lambda: ck.control_logits(dual),
                     lambda: ck.pick_tokens(dual)):
            with pytest.raises(ValueError):
                call()
            with torch.no_grad(), pytest.raises(ValueError):
                call()
        ck.int4_matvec(x, q, s, group_size=32)
        ck.pick_tokens(x)


def test_operands_that_want_a_gradient_are_refused():
    """Not x or the logits alone: a parameter among the other operands would get none."""
    import torch.autograd.forward_ad as fwd

    import sparse_graph_recurrent_gb300 as ck
    q, s, z = ck.int4_quantize(torch.randn(40, 64, device="cuda"), 32, symmetric=False)
    x = torch.randn(2, 64, device="cuda")
    product = dict(scales=s, zeros=z, bias=torch.randn(40, device="cuda"), out=torch.empty(2, 40, device="cuda"))
    rows = torch.rand(2, device="cuda") + 0.5
    control = dict(history=torch.zeros(2, 3, dtype=torch.int64, device="cuda"), repetition=rows, frequency=rows,
                   presence=rows, temperature=rows, bias=torch.randn(64, device="cuda"), out=torch.empty(2, 64, device="cuda"))
    calls = ((lambda **kw: ck.int4_matvec(x, q, group_size=32, **kw), product), (lambda **kw: ck.control_logits(x, **kw), control),
             (lambda **kw: ck.pick_tokens(x, **kw), control), (lambda **kw: ck.pick_tokens(x, seed=3, **kw), control))
    for call, operands in calls:
        want = call(**operands)
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
        for name, t in operands.items():
            if not t.is_floating_point():
                continue
            marked = {**operands, name: t.detach().clone().requires_grad_()}
            with pytest.raises(ValueError):
                call(**marked)
            with torch.no_grad():
                got = call(**marked)
            assert all(torch.equal(a, b) for a, b in zip(got if isinstance(got, tuple) else (got,), want)), name
            with fwd.dual_level(), pytest.raises(ValueError):
                call(**{**operands, name: fwd.make_dual(t.detach().clone(), torch.ones_like(t))})
