"""The compiled module's forms of the gated recurrence, clipping and beam search agree with
their Python forms, and what the module leaves is done or refused there."""
import pytest
import torch

from test_gpu_binding import both, same  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gated_both_ways(both):  # noqa: F811
    import sparse_graph_recurrent_gb300 as ck
    for T, dt in ((1, torch.float32), (40, torch.bfloat16), (3000, torch.float16)):
        x, gate = torch.randn(T, 3, 10, device="cuda").to(dt), torch.rand(T, 3, 10, device="cuda").to(dt)
        s, n = torch.randn(3, 10, device="cuda"), torch.tensor([T, 0, T // 2], device="cuda")
        for form in ("leak", "decay"):
            for kw in ({}, dict(state0=s), dict(state0=s, lengths=n), dict(state0=torch.randn(10, 3, device="cuda").t())):
                assert same(*both(lambda: ck.gated_recurrence(x, gate, form=form, **kw)))
                assert same(*both(lambda: ck.gated_recurrence(x[:, :, 1:7], gate[:1, :, 1:7], form=form,
                                                              **{k: v[:, 1:7] if k == "state0" else v for k, v in kw.items()})))
                a, b = both(lambda: ck.gated_recurrence_forward(x, gate, form=form, **kw))
                assert same(a, b)
                kw.pop("state0", None)
                for d, ds in ((x, s), (None, s), (x.transpose(0, 1).contiguous().transpose(0, 1), None)):
                    assert same(*both(lambda: ck.gated_recurrence_backward(x, gate, a[2], d, ds, form=form, **kw)))


def test_clip_both_ways(both):  # noqa: F811
    import sparse_graph_recurrent_gb300 as ck
    grads = [torch.randn(1000, device="cuda"), torch.randn(30, 7, device="cuda").half(), torch.randn(5, device="cuda").bfloat16()]

    def in_place(max_norm):
        mine = [g.clone() for g in grads]
        return (ck.clip_gradients(mine, max_norm), *mine)

    def apart(max_norm):
        out = tuple(torch.empty_like(g) for g in grads)
        return (ck.clip_gradients(tuple(grads), max_norm, out=out), *out)
    for max_norm in (1, 0.5, 1e9):
        assert same(*both(lambda: in_place(max_norm)))
        assert same(*both(lambda: apart(max_norm)))
    for some in (grads, grads[0], [None, grads[1]], [], (g for g in grads), [grads[0].view(10, 100).t()]):
        kind = list(some) if not isinstance(some, (list, torch.Tensor)) else some
        assert same(*both(lambda: ck.grad_norm(kind)))


def test_beams_both_ways(both):  # noqa: F811
    import sparse_graph_recurrent_gb300 as ck
    z, s = torch.randn(2, 3, 9000, device="cuda"), -torch.rand(2, 3, device="cuda")
    ended = torch.tensor([[True, False, False], [False, False, True]], device="cuda")
    for kw in ({}, dict(beams=5), dict(end_token=7), dict(ended=ended, end_token=0), dict(beams=1, ended=ended, end_token=8999)):
        assert same(*both(lambda: ck.beam_select(z, s, **kw)))
        assert same(*both(lambda: ck.beam_select(z.half()[..., 3:], s, **{**kw, **({"end_token": 5} if "end_token" in kw else {})})))
        assert same(*both(lambda: ck.beam_select(z.permute(1, 0, 2), s.t().repeat(1, 1), **{k: v for k, v in kw.items() if k == "beams"})))
    states = [torch.randn(2, 3, 50, device="cuda"), torch.randint(0, 5, (2, 3, 7), device="cuda"), ended]
    parents = torch.tensor([[2, 0, 0], [1, 1, 2]], device="cuda")
    assert same(*(tuple(r) for r in both(lambda: ck.reorder_states(states, parents))))
    assert same(*(tuple(r) for r in both(lambda: ck.reorder_states(tuple(states), parents[:, :2].contiguous()))))
    assert same(*both(lambda: ck.reorder_states(states[0], parents)))
    assert same(*both(lambda: ck.reorder_states(states[0].transpose(0, 1).contiguous().transpose(0, 1), parents)))

    def in_place():
        mine = [t.clone() for t in states]
        return tuple(ck.reorder_states(mine, parents, out=mine))
    assert same(*both(in_place))


def test_versions_rise_where_memory_is_written(both):  # noqa: F811
    import sparse_graph_recurrent_gb300 as ck

    def rises():
        g, o, s = (torch.randn(2, 3, 4, device="cuda") for _ in range(3))
        parents = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
        versions = [t._version for t in (g, o, s)]
        ck.clip_gradients([g], 0.1, out=[o])
        ck.clip_gradients([g], 0.1)
        ck.reorder_states([s], parents, out=[s])
        with torch.inference_mode():
            i = torch.randn(2, 3, 4, device="cuda")
            ck.clip_gradients([i], 0.1)
            ck.reorder_states([i], parents, out=[i])
        return all(t._version > v for t, v in zip((g, o, s), versions))
    assert both(rises) == (True, True)


def test_what_wants_a_gradient_is_refused():
    import torch.autograd.forward_ad as fwd

    import sparse_graph_recurrent_gb300 as ck
    x, s = torch.randn(2, 3, 8, device="cuda"), torch.randn(2, 3, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: ck.clip_gradients([dual], 1.0), lambda: ck.grad_norm([dual]), lambda: ck.beam_select(dual, s),
                     lambda: ck.reorder_states([dual], p), lambda: ck.reorder_states([x], p, out=[dual]),
                     lambda: ck.clip_gradients([x], 1.0, out=[dual])):
            with pytest.raises(ValueError):
                call()
        with pytest.raises((RuntimeError, NotImplementedError)):
            ck.gated_recurrence(dual, x)
    y = x.clone().requires_grad_()
    with torch.no_grad():
        ck.clip_gradients([y], 1.0)
        ck.reorder_states([y], p, out=[y])
    with pytest.raises(ValueError):
        ck.reorder_states([x], p, out=[y])
