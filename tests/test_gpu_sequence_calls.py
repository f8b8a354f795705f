"""Calls of the sequence operators that their documentation allows at its borders: one step of a
wider array, outputs laid out otherwise than the gradients, lists with nothing in them, views
that are conjugated or negated lazily, as many beams and tokens as there may be."""
import numpy as np
import pytest
import torch

import sequence_oracle as so
from test_gpu_beams import gathered
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


# -- views that are conjugated or negated when they are read ----------------------------------


def negated(t):
    """t, held as -t with a note to negate it."""
    n = torch._neg_view(t.neg())
    assert n.is_neg() and torch.equal(n, t)
    return n


def test_states_that_are_conjugated_or_negated_lazily():
    import sparse_graph_recurrent_gb300 as ck
    parents = torch.tensor([[1, 1, 0], [2, 0, 2]], device="cuda")
    z = torch.randn(2, 3, 40, dtype=torch.complex64, device="cuda")
    for state in (z.conj(), z.conj().imag, z.transpose(1, 2).contiguous().transpose(1, 2).conj(), negated(z.real.contiguous())):
        want = gathered(state.resolve_conj().resolve_neg(), parents)
        assert torch.equal(ck.reorder_states(state, parents).cpu(), want)
        assert all(torch.equal(t.cpu(), want) for t in ck.reorder_states([state, state], parents))
        out = torch.zeros(2, 3, 40, dtype=state.dtype, device="cuda")
        assert ck.reorder_states(state, parents, out=out) is out and torch.equal(out.cpu(), want)
    own = z.clone().conj()  # in its own place, and into one that is noted alike
    want = gathered(own.resolve_conj(), parents)
    like = torch.zeros_like(z).conj()
    ck.reorder_states(own, parents, out=like)
    assert like.is_conj() and torch.equal(like.resolve_conj().cpu(), want)
    ck.reorder_states(own, parents, out=own)
    assert own.is_conj() and torch.equal(own.resolve_conj().cpu(), want)
    with pytest.raises(ValueError):
        ck.reorder_states(z, parents, out=torch.zeros_like(z).conj())


@pytest.mark.parametrize("dtype", list(TYPES))
def test_operands_that_are_negated_lazily(dtype):
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(40, 3, 8, dtype, "leak")
    plain = ck.gated_recurrence_forward(d["x"], d["gate"], d["state0"])
    want = ck.gated_recurrence_backward(d["x"], d["gate"], plain[2], d["d_out"], d["d_state"])
    for name in ("x", "gate", "state0", "d_out", "d_state"):
        n = {**d, name: negated(d[name])}
        got = ck.gated_recurrence_forward(n["x"], n["gate"], n["state0"])
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
        assert all(torch.equal(a, b) for a, b in zip(ck.gated_recurrence(n["x"], n["gate"], n["state0"]), plain))
        got = ck.gated_recurrence_backward(n["x"], n["gate"], got[2], n["d_out"], n["d_state"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    z, s = d["x"][:2].transpose(1, 2).contiguous(), -torch.rand(2, 8, device="cuda")
    want = ck.beam_select(z, s)
    for args in ((negated(z), s), (z, negated(s))):
        assert all(torch.equal(a, b) for a, b in zip(ck.beam_select(*args), want))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_clipping_of_what_is_negated_lazily(dtype):
    import sparse_graph_recurrent_gb300 as ck
    g = torch.randn(300, device="cuda").to(TYPES[dtype])
    want = torch.empty_like(g)
    norm = ck.clip_gradients([g], 0.5, out=[want])
    for a in (g, negated(g)):
        for b in (torch.empty_like(g), torch._neg_view(torch.empty_like(g))):
            assert torch.equal(ck.clip_gradients([a], 0.5, out=[b]), norm)
            assert torch.equal(b.resolve_neg(), want) and torch.equal(a.resolve_neg(), g)
    own = negated(g)
    assert torch.equal(ck.clip_gradients([own], 0.5), norm) and torch.equal(own.resolve_neg(), want)


def test_readout_operands_that_are_negated_lazily():
    """The readout's operators look at their operands the same way."""
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(3, 64, device="cuda")
    assert torch.equal(ck.dropout(negated(x), 0.3, 5), ck.dropout(x, 0.3, 5))
    w = torch.randn(40, 64, device="cuda")
    q = ck.int4_quantize(w, 32)
    assert all(torch.equal(a, b) for a, b in zip(ck.int4_quantize(negated(w), 32)[:2], q[:2]))
    bias = torch.randn(40, device="cuda")
    want = ck.int4_matvec(x, *q, bias, 32)
    for args in ((negated(x), *q, bias, 32), (x, q[0], negated(q[1]), q[2], bias, 32), (x, *q, negated(bias), 32)):
        assert torch.equal(ck.int4_matvec(*args), want)
    with pytest.raises(ValueError):
        ck.int4_matvec(x, *q, bias, 32, out=torch._neg_view(want.clone()))
    heat, extra = torch.rand(3, device="cuda") + 0.5, torch.randn(64, device="cuda")
    want = ck.control_logits(x, bias=extra, temperature=heat)
    for z, b, t in ((negated(x), extra, heat), (x, negated(extra), heat), (x, extra, negated(heat))):
        assert torch.equal(ck.control_logits(z, bias=b, temperature=t), want)
    assert torch.equal(ck.pick_tokens(negated(x)), ck.pick_tokens(x))
    with pytest.raises(ValueError):
        ck.control_logits(x, out=torch._neg_view(want.clone()))


# -- selection -------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,K,V", [("float32", 64, 4_600_000), ("float32", 64, 16_777_215), ("bfloat16", 64, 9_400_000)])
def test_as_many_beams_and_tokens_as_there_may_be(dtype, K, V):
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn(1, K, V, generator=g, device="cuda").to(TYPES[dtype])
    scores = -torch.rand(1, K, generator=g, device="cuda")
    got = ck.beam_select(logits, scores)
    base = torch.stack([torch.logsumexp(z.double(), 0) for z in logits[0]])
    top = torch.topk(logits[0], 64, dim=1)
    for r in range(K):
        k, v = int(got[1][0, r]), int(got[2][0, r])
        want = float(scores[0, k]) + float(logits[0, k, v]) - float(base[k])
        assert abs(float(got[0][0, r]) - want) <= so.beam_score_off(V) + abs(want) * so.U32
    all_of_them = scores[0].double()[:, None] + top.values.double() - base[:, None]
    best = torch.topk(all_of_them.flatten(), 64).values
    assert (got[0][0].double() - best).abs().max() <= so.beam_score_off(V) + 2 * so.U32 * float(best.abs().max())


# -- calls in a row, each on what the one before has written -----------------------------------


@pytest.mark.parametrize("n", [300, 70_000, 3_000_000])
def test_clipped_again_and_again(n):
    """The kernels of a call take their places while those before end; what they read was written
    by the call before, at the same places."""
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator().manual_seed(n)
    start = [torch.randn(n, generator=g).cuda(), torch.randn(n // 3, generator=g).bfloat16().cuda()]
    limits = [300.0, 200.0, 30.0, 10.0, 9.0, 1.0, 0.7, 0.3]

    def run(wait):
        grads, norms = [t.clone() for t in start], []
        for limit in limits:
            norms.append(ck.clip_gradients(grads, limit))
            if wait:
                torch.cuda.synchronize()
        return grads, norms
    want, norms = run(True)
    for _ in range(20):
        got, n2 = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got + n2, want + norms))


def test_searched_again_and_again():
    """Scores, parents, ends and lengths that the kernels before have just written."""
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator().manual_seed(3)
    embed, gates = (torch.randn(50, 64, generator=g).cuda() for _ in range(2))
    read = torch.randn(64, 50, generator=g).cuda()

    def run(wait):
        torch.cuda.synchronize()
        state = torch.zeros(3, 8, 64, device="cuda")
        scores, ended = torch.zeros(3, 8, device="cuda"), torch.zeros(3, 8, dtype=torch.bool, device="cuda")
        all_of_it = []
        for _ in range(12):
            logits = (state.view(24, 64) @ read).view(3, 8, 50)
            scores, parents, tokens, ended = ck.beam_select(logits, scores, ended, 7)
            ck.reorder_states(state, parents, out=state)
            out, new = ck.gated_recurrence(embed[tokens.view(-1)][None], gates[tokens.view(-1)][None], state.view(24, 64),
                                           (~ended).long().view(-1))
            state = new.view(3, 8, 64)
            all_of_it += [scores, parents, tokens, ended, out, state]
            if wait:
                torch.cuda.synchronize()
        return all_of_it
    want = run(True)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))


# -- decays beyond 1 -------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,B,N", [(600, 1, 40), (2000, 3, 4000), (2000, 1, 70), (1100, 2, 601), (9000, 1, 33), (40_000, 1, 6)])
def test_decays_whose_products_leave_32_bits(T, B, N, dtype):
    """States that stay inside 32 bits although the products of decays do not: 0 where nothing has
    come in yet, or begun low.  Steps one after another give them; however they are cut does too."""
    import sparse_graph_recurrent_gb300 as ck
    g, dt = torch.Generator().manual_seed(T), TYPES[dtype]
    gate = torch.full((T, B, N), 2.0, dtype=dt, device="cuda")
    x, d_out = torch.zeros_like(gate), torch.zeros_like(gate)
    x[-20:] = torch.randn(20, B, N, generator=g).cuda()
    d_out[:20] = torch.randn(20, B, N, generator=g).cuda()
    out, state, kept = ck.gated_recurrence_forward(x, gate, None, None, "decay")
    assert not out[:-20].any()
    want, off = so.gated(host(x[-20:]), host(gate[-20:]), None, None, "decay")
    so.within(host(out[-20:]), want["out"], off["out"], dtype)
    so.within(host(state), want["state"], off["state"])
    dx, dgate, dstate0 = ck.gated_recurrence_backward(x, gate, kept, d_out, None, None, "decay")
    want, off = so.gated(host(x[:20]), host(gate[:20]), None, None, "decay", host(d_out[:20]))
    so.within(host(dx[:20]), want["dx"], off["dx"], dtype)
    so.within(host(dstate0), want["dstate0"], off["dstate0"])
    assert not dx[20:].any() and not dgate.any()
    # from 2^-100 up by more than 32 bits hold, down again, and so on: powers of 2, and exact
    t = torch.arange(T) % 400
    power = torch.where(t < 200, t + 1, 399 - t).double() - 100
    powers = torch.exp2(power).to(dt).view(T, 1, 1).expand(T, B, N).cuda()
    gate = torch.where(t < 200, 2.0, 0.5).to(dt).view(T, 1, 1).expand(T, B, N).contiguous().cuda()
    zero = torch.zeros_like(gate)
    start = torch.full((B, N), 2.0 ** -100, device="cuda")
    out, state, kept = ck.gated_recurrence_forward(zero, gate, start, None, "decay")
    assert torch.equal(out, powers)
    last = torch.full((B, N), 2.0 ** -float(power[-1]), device="cuda")
    dx, dgate, dstate0 = ck.gated_recurrence_backward(zero, gate, kept, None, last, None, "decay")
    assert (dstate0 == 2.0 ** 100).all()
    assert torch.equal(dx, torch.exp2(-power).to(dt).view(T, 1, 1).expand(T, B, N).cuda())
    # the same where the last sequence ends before the others
    lengths = torch.full((B,), T, device="cuda")
    lengths[-1] = T - 137
    gate[T - 137:, -1] = float("nan")
    out, state, kept = ck.gated_recurrence_forward(zero, gate, start, lengths, "decay")
    assert torch.equal(out[:, :-1], powers[:, :-1]) and torch.equal(out[:T - 137, -1], powers[:T - 137, -1])
    assert not out[T - 137:, -1].any() and (state[-1] == 2.0 ** float(power[T - 138])).all()
    last[-1] = 2.0 ** -float(power[T - 138])
    dx, dgate, dstate0 = ck.gated_recurrence_backward(zero, gate, kept, None, last, lengths, "decay")
    assert (dstate0 == 2.0 ** 100).all() and not dx[T - 137:, -1].any()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,B,N", [(300, 2, 30), (2000, 1, 70), (9000, 1, 33)])
def test_large_states(T, B, N, dtype):
    """States of 2^30 and more, with nothing coming in at first, for a while, and at last."""
    d = inputs(T, B, N, dtype, "decay", seed=T)
    for name in ("x", "d_out"):
        d[name] *= 2.0 ** 30
        for lo, hi in ((0, 1), (4, 5), (9, 10)):
            d[name][T * lo // 10:T * hi // 10] = 0
    d["state0"] = None
    d["gate"] = (d["gate"].float() * 0.3 + 0.7).to(TYPES[dtype])
    check(d, "decay", dtype)


@pytest.mark.parametrize("T", [700, 9000])
def test_an_infinite_input_reaches_what_it_would_step_by_step(T):
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(T, 2, 33, "float32", "decay")
    d["x"][T // 3, 0, 5] = float("inf")
    d["x"][T // 2, 1, 7] = float("nan")
    d["gate"][2 * T // 3, 0, 5] = 0.0  # infinity times 0
    out, state, kept = ck.gated_recurrence_forward(d["x"], d["gate"], d["state0"], None, "decay")
    h = d["state0"].double()
    for t in range(T):
        h = d["gate"][t].double() * h + d["x"][t].double()
        if t in (0, T // 3, T // 2, 2 * T // 3 - 1, 2 * T // 3, T - 1):
            assert torch.equal(out[t].isnan(), h.isnan()) and torch.equal(out[t].isinf(), h.isinf())
    d["d_out"][T // 2, 1, 9] = float("inf")
    dx = ck.gated_recurrence_backward(d["x"], d["gate"], kept, d["d_out"], d["d_state"], None, "decay")[0]
    assert dx[:T // 2 + 1, 1, 9].isinf().all() and dx[T // 2 + 1:].isfinite().all()


@pytest.mark.parametrize("T,B,N", [(2000, 3, 4000), (2000, 1, 70), (9000, 1, 33)])
def test_a_large_input_that_fades(T, B, N):
    """2^100 comes in, and is halved and doubled again and again."""
    import sparse_graph_recurrent_gb300 as ck
    t = torch.arange(T) % 500
    for at in (0, 37, T // 2, T - 300):
        x = torch.zeros(T, B, N, device="cuda")
        x[at] = 2.0 ** 100
        n = (torch.arange(T) - at) % 400
        gate = torch.where((n > 0) & (n <= 200), 0.5, 2.0)
        gate[:at + 1] = 1
        power = 100 - torch.where(n <= 200, n, 400 - n).double()
        want = torch.where(torch.arange(T) < at, 0.0, torch.exp2(power)).float().view(T, 1, 1).expand(T, B, N).cuda()
        gate = gate.view(T, 1, 1).expand(T, B, N).contiguous().cuda()
        assert torch.equal(ck.gated_recurrence(x, gate, None, None, "decay")[0], want)
        # and the other way round: a gradient
        x, gate = x.flip(0), torch.cat((gate[1:], gate[:1] * 0 + 1)).flip(0)
        zero = torch.zeros_like(x)
        kept = ck.gated_recurrence_forward(zero, gate, None, None, "decay")[2]
        assert torch.equal(ck.gated_recurrence_backward(zero, gate, kept, x, None, None, "decay")[0], want.flip(0))


# -- reordering ------------------------------------------------------------------------------


def test_two_halves_of_one_array():
    """States and where they go side by side in one array, however its axes lie."""
    import sparse_graph_recurrent_gb300 as ck
    parents = torch.tensor([[1, 1, 0, 2], [2, 0, 2, 3], [3, 3, 1, 0]], device="cuda")
    whole = lambda *n: torch.randn(*n, device="cuda")  # noqa: E731
    for both in (whole(3, 2, 4, 33).unbind(1), whole(2, 3, 4, 33).unbind(0), whole(3, 4, 2, 33).unbind(2),
                 [t.transpose(0, 1) for t in whole(4, 2, 3, 33).unbind(1)], whole(3, 5, 2, 4, 8).unbind(2)[0].unbind(1)[1:3],
                 whole(3, 8, 33).split(4, 1), whole(3, 4, 66).split(33, 2)):
        a, b = both
        for source, to in ((a, b), (b, a)):
            if source.shape[1] != 4:
                continue
            want, keep = gathered(source, parents), source.clone()
            assert ck.reorder_states(source, parents, out=to) is to
            assert torch.equal(to.cpu(), want) and torch.equal(source, keep)
    # fewer go on than there were
    line = whole(3, 7, 20)
    want = gathered(line[:, :4], parents[:, :3])
    ck.reorder_states(line[:, :4], parents[:, :3], out=line[:, 4:])
    assert torch.equal(line[:, 4:].cpu(), want)
    line = whole(3, 7, 20)
    for source, to in ((line[:, :4], line[:, 3:7]), (line[:, :4, :12], line[:, :4, 8:]), (line[:, :4], line[:, 1:5])):
        with pytest.raises(RuntimeError):
            ck.reorder_states(source, parents, out=to)


def test_parents_that_are_a_state_too():
    import sparse_graph_recurrent_gb300 as ck
    parents = torch.tensor([[1, 1, 0], [2, 0, 2]], device="cuda")
    assert torch.equal(ck.reorder_states(parents, parents).cpu(), gathered(parents, parents))
    keep = parents.clone()
    for states, out in (([parents], [parents]), ([keep], [parents])):
        with pytest.raises(RuntimeError):
            ck.reorder_states(states, parents, out=out)
    assert torch.equal(keep, parents)


def test_strided_tensors_that_share_memory():
    import sparse_graph_recurrent_gb300 as ck
    w, to = torch.randn(8, 12, device="cuda"), torch.zeros(8, 12, device="cuda")
    for grads in ([w[:, :3], w[:, 2:5]], [w[:, ::2], w[:, ::3]], [w[::2], w[:3]], [w[:, :5], w], [w.t()[:3], w[:2]],
                  [w[:, 0], w[0]], [w[:, ::2], w[:, 1:3]]):
        keep = w.clone()
        with pytest.raises((ValueError, RuntimeError)):
            ck.clip_gradients(grads, 0.5)
        assert torch.equal(w, keep)
        with pytest.raises((ValueError, RuntimeError)):  # read in one, written in another
            ck.clip_gradients([grads[0], to[:grads[1].shape[0], :grads[1].shape[1]] if grads[1].dim() == 2 else to[0, :grads[1].shape[0]]],
                              0.5, out=[torch.empty_like(grads[0]), grads[1]])
        assert torch.equal(w, keep)
        ck.grad_norm(grads)  # reading is fine
    # side by side is fine
    for cut in (lambda t: [t[:, ::2], t[:, 1::2]], lambda t: [t[:, :3], t[:, 3:7], t[:, 7:]], lambda t: [t[::2, 1::2], t[1::2]],
                lambda t: [t[:, 0], t[:, 1], t[:4, 2:], t[4:, 2:]], lambda t: [t.t()[:5], t[:, 5:]],
                lambda t: [t[:, ::2], t[:, 1:2], t[:, 3::2]], lambda t: [t[:, :4].t(), t[:, 4:8], t[:, 11]]):
        t, o = w.clone(), torch.full_like(w, 7)
        parts = [host(p) for p in cut(t)]
        norm, factor = so.clip(parts, 0.5)
        ck.clip_gradients(cut(t), 0.5, out=cut(o))
        assert torch.equal(t, w)
        got = ck.clip_gradients(cut(t), 0.5)
        assert abs(float(got) - norm) <= NORM_OFF * norm
        for p, q, v in zip(cut(t), cut(o), parts):
            assert torch.equal(p, q)
            so.within(host(p), v * factor, np.abs(v * factor) * FACTOR_OFF)
    with pytest.raises(ValueError):
        ck.clip_gradients([w[0]], 0.5, out=[to[:1, :1].expand(1, 12)[0]])
    # dense, and in another order than its gradient
    c = torch.zeros(6, 4, device="cuda")
    for grads, out in (([w[:4, :6].contiguous(), c.view(-1)[3:9]], [c.t(), torch.zeros(6, device="cuda")]),
                       ([w[:4, :6].contiguous(), w[7]], [c.t(), c.view(-1)[12:]]), ([c.view(4, 6)], [c.t()])):
        with pytest.raises((ValueError, RuntimeError)):
            ck.clip_gradients(grads, 0.5, out=out)


@pytest.mark.parametrize("max_norm", [1.0, 1e38, 1e39, 1e300])
def test_an_infinite_norm_gives_a_factor_of_0(max_norm):
    import sparse_graph_recurrent_gb300 as ck
    for big in (3e38, float("inf")):  # (the root of two squares of 3e38 is beyond 32 bits too)
        g = torch.full((5000,), big, device="cuda")
        rest = torch.randn(77, device="cuda")
        assert float(ck.clip_gradients([g, rest], max_norm)) == float("inf")
        assert not rest.any() and (not g.any() if big < float("inf") else g.isnan().all())


def test_no_limit_changes_nothing():
    import sparse_graph_recurrent_gb300 as ck
    for big in (1.0, 3e38, float("inf")):
        g = torch.full((5000,), big, device="cuda")
        out = torch.empty_like(g)
        ck.clip_gradients([g], float("inf"), out=[out])
        assert torch.equal(g, out)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -80, 2.0 ** 70])
def test_the_norm_of_billions(scale):
    """A number whose squares' sum is rounded the same way again and again, where a thread adds up
    a thousand chunks of it: a sum of 32 bits that takes in all of them is off by 128 half steps.
    The bound is of an element's square, 32 additions in a chunk and 32 chunks in a row, in half
    steps, halved by the root, which is rounded."""
    import sparse_graph_recurrent_gb300 as ck
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 4 * sms * 1050 * 4096
    c = float.fromhex("0x1.ef60e80000000p0") * scale
    g = torch.full((n,), c, device="cuda")
    want = c * float(n) ** 0.5
    assert abs(float(ck.grad_norm(g)) - want) <= ((1 + 32 + 32) / 2 + 1) * so.U32 * want
    half = 0.5 * want
    assert abs(float(ck.clip_gradients(g, half)) - want) <= ((1 + 32 + 32) / 2 + 1) * so.U32 * want
    got = c * half / (want + 1e-6)  # (by the definition: far from half of c where the norm is small)
    assert abs(float(g[0]) - got) <= 40 * so.U32 * got and (g == g[0]).all()
