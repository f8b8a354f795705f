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
