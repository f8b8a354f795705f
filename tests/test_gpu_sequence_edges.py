"""Where the gated recurrence, clipping and beam search could go wrong at the seams: rows that
begin anywhere, candidates in few hands, numbers at the ends of their range, and calls in a
row whose kernels overlap."""
import numpy as np
import pytest
import torch

import sequence_oracle as so
from test_gpu_beams import check as check_beams
from test_gpu_beams import make as make_beams
from test_gpu_clip import FACTOR_OFF, NORM_OFF
from test_gpu_gated import TYPES, check, host, inputs

pytestmark = pytest.mark.gpu


# -- gated recurrence ------------------------------------------------------------------------


def moved(t, offset):
    """A copy of t that begins `offset` elements behind a multiple of 512 bytes."""
    line = torch.full((t.numel() + offset + 8,), float("nan"), dtype=t.dtype, device="cuda")
    return line[offset:offset + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,N", [(1, 64), (2, 33), (3, 43), (1, 201), (5, 26), (2, 100), (3, 44), (7, 1)])
def test_rows_that_begin_anywhere(B, N, dtype, form):
    for T, offsets in ((9, (1, 1, 1)), (25, (3, 3, 3)), (25, (0, 8, 16)), (130, (5, 5, 5)), (18, (0, 1, 2)), (18, (2, 2, 6))):
        d = inputs(T, B, N, dtype, form, seed=T + N, lengths=T != 25)
        for name, offset in zip(("x", "gate", "d_out"), offsets):
            d[name] = moved(d[name], offset)
        check(d, form, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_what_lies_around_the_outputs_stays(dtype):
    """Through the C entries, with outputs that begin at an odd place."""
    from sparse_graph_recurrent_gb300 import _ck
    for T, B, N in ((11, 1, 65), (16, 3, 22), (40, 2, 8)):
        d = inputs(T, B, N, dtype, "leak", lengths=True)
        kept_bytes, need = _ck.ck_gated_sizes(T, B, N)
        n = T * B * N
        lines = [torch.full((n + 10,), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(3)]
        state, kept = torch.empty(B, N, device="cuda"), torch.empty(kept_bytes // 4, device="cuda")
        ws = torch.empty(need // 8 + 1, dtype=torch.int64, device="cuda")
        e = lines[0].element_size()
        for at in (0, 1, 3):
            args = dict(x=d["x"].data_ptr(), gate=d["gate"].data_ptr(), dtype=_ck.DTYPES[TYPES[dtype]], form=0, T=T, B=B, N=N,
                        x_step=B * N, x_row=N, gate_step=B * N, gate_row=N, lengths=d["lengths"].data_ptr(),
                        kept=kept.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=need)
            _ck.ck_gated_forward(_ck.GatedCall(state0=d["state0"].data_ptr(), out=lines[0].data_ptr() + at * e,
                                               state=state.data_ptr(), **args))
            _ck.ck_gated_backward(_ck.GatedCall(d_out=d["d_out"].data_ptr(), d_out_step=B * N, d_out_row=N,
                                                d_state=d["d_state"].data_ptr(), dx=lines[1].data_ptr() + at * e,
                                                dgate=lines[2].data_ptr() + at * e, **args))
            want, off = so.gated(host(d["x"]), host(d["gate"]), host(d["state0"]), d["lengths"].cpu().numpy(), "leak",
                                 host(d["d_out"]), host(d["d_state"]))
            for line, name in zip(lines, ("out", "dx", "dgate")):
                so.within(host(line[at:at + n]).reshape(T, B, N), want[name], off[name], dtype)
                assert (line[:at] == 7).all() and (line[at + n:] == 7).all()
                line.fill_(7)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,B,N", [(31, 1, 4), (32, 1, 4), (33, 1, 4), (2047, 1, 3), (129, 16, 1024)])
def test_steps_cut_into_parts(T, B, N, dtype):
    """Around the numbers of steps at which another warp, or another CTA, takes a part."""
    check(inputs(T, B, N, dtype, "decay", seed=T, lengths=B > 1), "decay", dtype)
    check(inputs(T, B, N, dtype, "leak", seed=T), "leak", dtype)


@pytest.mark.parametrize("form", ["leak", "decay"])
def test_many_rows_of_whole_pairs(form):
    """Enough of them that 32-bit rows at multiples of 8 bytes are taken as they lie."""
    check(inputs(131, 2, 16_141, "float32", form, seed=1, lengths=True), form, "float32")


def test_a_gradient_of_what_was_not_given():
    """d_out or d_state alone, at rows that begin anywhere."""
    import sparse_graph_recurrent_gb300 as ck
    for T, N, dt in ((37, 33, torch.float16), (2100, 3, torch.float32), (64, 64, torch.bfloat16)):
        x, gate = (moved(torch.randn(T, 1, N, device="cuda").to(dt), 1) for _ in range(2))
        _, _, kept = ck.gated_recurrence_forward(x, gate)
        d, ds = torch.randn(T, 1, N, device="cuda").to(dt), torch.randn(1, N, device="cuda")
        zero, none = torch.zeros_like(d), torch.zeros_like(ds)
        for some, all_ in (((None, ds), (zero, ds)), ((d, None), (d, none)), ((None, None), (zero, none))):
            got, want = (ck.gated_recurrence_backward(x, gate, kept, *a) for a in (some, all_))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_too_many_nodes_are_refused():
    from sparse_graph_recurrent_gb300 import _ck
    with pytest.raises(_ck.CKError):
        _ck.ck_gated_sizes(1, 2 ** 14, 2 ** 14 + 1)
    assert _ck.ck_gated_sizes(1, 2 ** 14, 2 ** 14)[0] == 4 * 2 ** 28


# -- clipping --------------------------------------------------------------------------------


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-8, 1e22, 3e37])
def test_a_run_of_another_size_beside_ordinary_ones(scale):
    """CTAs whose squares leave 32 bits, others whose do not, and zeros."""
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator().manual_seed(1)
    some = [torch.randn(n, generator=g).cuda() for n in (500_000, 3, 700_001)]
    some[0] *= scale
    some.insert(1, torch.zeros(300_000, device="cuda"))
    some.append(torch.full((100_000,), -0.0, device="cuda"))
    for grads in (some, some[:2], some[1:2], [some[1], some[-1]]):
        want = [host(t) for t in grads]
        norm, factor = so.clip(want, 0.5)
        got = ck.grad_norm(grads)
        if norm > np.finfo(np.float32).max:  # a norm that 32 bits do not hold is infinite, the factor 0
            norm, factor = np.inf, 0.0
            assert float(got) == norm
        else:
            assert abs(float(got) - norm) <= NORM_OFF * norm
        out = [torch.empty_like(t) for t in grads]
        assert torch.equal(ck.clip_gradients(grads, 0.5, out=out), got)
        for o, w in zip(out, want):
            so.within(host(o), w * factor, np.abs(w * factor) * FACTOR_OFF)


def test_lists_that_lie_in_any_order():
    """Overlaps are found, and only overlaps, wherever inputs and outputs lie to each other."""
    import sparse_graph_recurrent_gb300 as ck
    line = torch.randn(100_000, device="cuda")
    half = line.view(torch.float16)
    cut = lambda t, at, n=50: t[at:at + n]  # noqa: E731
    order = torch.randperm(400, generator=torch.Generator().manual_seed(2)).tolist()
    grads = [cut(line, 100 * i) for i in order]
    out = [cut(line, 100 * i + 50) for i in order]
    want = [t.clone() for t in grads]
    norm = ck.clip_gradients(grads, 1e9, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and float(norm) > 0
    far = [torch.empty(50, device="cuda") for _ in order]
    ck.clip_gradients(grads, 1e9, out=far)
    for bad in (lambda: ck.clip_gradients(grads, 1.0, out=out[:399] + [cut(line, 100 * order[0] + 99)]),
                lambda: ck.clip_gradients(grads, 1.0, out=out[:399] + [cut(line, 100 * order[7] + 49)]),
                lambda: ck.clip_gradients(grads + [cut(half, 20)], 1.0, out=out + [cut(half, 200 * order[3] + 198)]),
                lambda: ck.clip_gradients(grads + [cut(half, 200 * order[5])], 1.0)):
        with pytest.raises(RuntimeError):
            bad()


# -- beam search -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_candidates_in_few_hands(dtype):
    """All that is left of the vocabulary lies where one lane, or one thread, looks."""
    V = 40_000
    logits, scores = make_beams(2, 3, V, dtype, seed=9)
    e = 16 // logits.element_size()
    token = torch.arange(V, device="cuda")
    thread = token // e % 256
    for keep in (thread % 32 == 5, thread == 77, (thread % 32 < 3) & (token < 20_000), thread // 32 == 6):
        check_beams(logits.masked_fill(~keep, -float("inf")), scores, beams=16)
    # one beam far ahead, whose best lie in all of its slices; and one whose best lie in one
    scores[:, 1] += 40
    check_beams(logits, scores, beams=32)
    logits[:, 1, :3000] += 20
    for beams in (1, 7, 32, 33, 64):
        check_beams(logits, scores, beams=beams)


@pytest.mark.parametrize("scale", [300.0, 1e3, 3e4, 1e6, 1e30])
def test_logits_of_any_size(scale):
    logits, scores = make_beams(2, 4, 9001, torch.float32, seed=3)
    check_beams(logits * scale, scores, beams=8)
    check_beams(logits - scale, scores, beams=8)
    check_beams(logits * scale, scores * scale, beams=8)
    if scale < 1e4:
        check_beams((logits * scale).half(), scores, beams=8)


@pytest.mark.parametrize("K,V", [(8, 8192), (4, 8193), (8, 8193), (9, 100), (2, 32768), (2, 32769), (1, 65537), (33, 16384),
                                 (64, 70_000)])
def test_around_the_kernels_borders(K, V):
    """One launch or two, few lists or many."""
    for dtype in (torch.float32, torch.float16):
        logits, scores = make_beams(2, K, V, dtype, seed=K)
        ended = torch.rand(2, K, generator=torch.Generator().manual_seed(V)) < 0.2
        check_beams(logits, scores, ended.cuda(), V - 1, beams=min(16, K * 2))


def test_a_vocabulary_of_millions():
    """More lists than the second kernel looks at side by side."""
    logits, scores = make_beams(1, 2, 5_000_003, torch.float16, seed=2)
    check_beams(logits, scores, beams=5)
    logits, scores = make_beams(1, 1, 4_500_001, torch.float32, seed=2)
    check_beams(logits, scores, beams=32)


# -- offsets that pass 32 bits ---------------------------------------------------------------


def test_states_beyond_32_bits():
    """More than 2^31 elements, whole and by rows far apart; a state that has settled tells
    whether each step found its own."""
    import sparse_graph_recurrent_gb300 as ck
    T, N = 66_000, 32_771
    x = torch.randn(1, 1, N, device="cuda").bfloat16()
    gate = torch.full((1, 1, 1), 0.5, device="cuda", dtype=torch.bfloat16)
    full = lambda t: t.expand(T, 1, N)  # noqa: E731
    out, state, kept = ck.gated_recurrence_forward(full(x), full(gate), form="decay")
    assert torch.equal(state, x[0].float() * 2)  # sums of 1, 1/2, ... to the last place
    settled = (x[0, 0].float() * 2).bfloat16()
    for i in range(64, T, 6000):
        assert (out[i:i + 6000] == settled).all()
    dx, dgate, d0 = ck.gated_recurrence_backward(full(x), full(gate), kept, out, form="decay")
    # g settles at twice d_out, its product with a settled state at 8 x^2
    want = (out[100, 0].float() * 2).bfloat16()
    product = (out[100, 0].float() * 2) * (x[0, 0].float() * 2)
    for i in range(100, T - 100, 6000):
        n = min(6000, T - 100 - i)
        assert (dx[i:i + n] == want).all()
        assert ((dgate[i:i + n].float() - product).abs() <= product.abs() * 2.0 ** -7).all()
    last = out[-1].clone()
    del out, dx, dgate, kept
    wide = torch.zeros(3, 1, 2 ** 30 + 8, device="cuda", dtype=torch.bfloat16)  # rows far apart
    far = wide[:, :, 4:4 + N]
    far.copy_(x.expand(3, 1, N))
    a, b = (ck.gated_recurrence(v, full(gate)[:3], form="decay") for v in (far, x.expand(3, 1, N).contiguous()))
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and torch.equal(last[0], settled)


def test_gradients_beyond_32_bits():
    import sparse_graph_recurrent_gb300 as ck
    n = 2 ** 31 + 12_345
    g = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    g[-1] = 1024.0
    want = np.sqrt((n - 1) * 0.25 + 1024.0 ** 2)
    norm = ck.clip_gradients([g[:3], g[3:]], want / 2)
    assert abs(float(norm) - want) <= NORM_OFF * want
    assert float(g[-1]) == 512 and float(g[0]) == 0.25 and (g[-2 ** 20:-1] == 0.25).all() and (g[2 ** 30:2 ** 30 + 9] == 0.25).all()


def test_beams_states_beyond_32_bits():
    import sparse_graph_recurrent_gb300 as ck
    t = torch.zeros(2, 2, 2 ** 30 + 3, dtype=torch.uint8, device="cuda")
    t[0, 0], t[0, 1], t[1, 0], t[1, 1] = 1, 2, 3, 4
    t[1, 1, -1] = 5
    parents = torch.tensor([[1, 1], [1, 0]], device="cuda")
    got = ck.reorder_states(t, parents)
    assert (got[0] == 2).all() and (got[1, 0, :-1] == 4).all() and got[1, 0, -1] == 5 and (got[1, 1] == 3).all()
    ck.reorder_states([t], parents, out=[t])
    assert torch.equal(t, got)


# -- calls in a row --------------------------------------------------------------------------


def test_kernels_that_overlap_wait_for_what_they_read():
    """Many steps without a pause give what steps with a pause after every call give."""
    import sparse_graph_recurrent_gb300 as ck
    B, K, V, N = 3, 4, 9000, 700
    g = torch.Generator().manual_seed(11)
    embed, gates = (torch.randn(V, N, generator=g).cuda() for _ in range(2))
    read = (torch.randn(N, V, generator=g) * 0.3).cuda()

    def steps(pause):
        state, scores = torch.zeros(B, K, N, device="cuda"), torch.zeros(B, K, device="cuda")
        scores[:, 1:] = -float("inf")
        text = torch.zeros(B, K, 40, dtype=torch.int64, device="cuda")
        rest = (lambda: torch.cuda.synchronize()) if pause else (lambda: None)  # noqa: E731
        got = []
        for i in range(40):
            logits = (state.view(B * K, N) @ read).view(B, K, V)
            rest()
            scores, parents, tokens, _ = ck.beam_select(logits, scores)
            rest()
            ck.reorder_states([state, text], parents, out=[state, text])
            rest()
            text[..., i] = tokens
            t = tokens.view(-1)
            state = ck.gated_recurrence(embed[t].unsqueeze(0), gates[t].unsqueeze(0), state.view(B * K, N))[1].view(B, K, N)
            rest()
            norm = ck.clip_gradients([state, scores], 50.0)
            rest()
            got.append(norm)
        return state, scores, text, torch.stack(got)
    want = steps(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))


def test_a_layer_trained_in_a_captured_step():
    """Recurrence, its gradients, their clipping and an update, captured and replayed, are the
    same calls made one after another."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    T, B, N = 70, 3, 45
    g = torch.Generator().manual_seed(5)
    x, d_out = (torch.randn(T, B, N, generator=g).cuda() for _ in range(2))
    n = torch.tensor([70, 0, 33], device="cuda")

    def step(gate):
        out, state, kept = ck.gated_recurrence_forward(x, gate, lengths=n)
        dx, dgate, _ = ck.gated_recurrence_backward(x, gate, kept, d_out, state, lengths=n)
        norm = ck.clip_gradients([dx, dgate], 1.0)
        _ck.ck_sgd_update(gate, dgate, 0.5)
        return norm, out
    eager = torch.randn(T, B, N, generator=torch.Generator().manual_seed(6)).cuda()
    captured = eager.clone()
    step(captured.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(captured)
    for _ in range(4):
        want = step(eager)
        graph.replay()
        assert torch.equal(eager, captured) and all(torch.equal(a, b) for a, b in zip(got, want))


def handed_over(x, gate, read, scores, other, pause=lambda: None):
    """Each call's operands come from the other stream, which waits for the call before."""
    import sparse_graph_recurrent_gb300 as ck
    here = torch.cuda.current_stream()

    def there(make):
        other.wait_stream(here)
        with torch.cuda.stream(other):
            made = make()
        here.wait_stream(other)
        pause()
        return made
    B, K = scores.shape
    state = torch.zeros(B * K, x.shape[2], device="cuda")
    for _ in range(8):
        d = there(lambda: x + state.sum() * 1e-3)
        out, state, kept = ck.gated_recurrence_forward(d, gate, state)
        pause()
        g = there(lambda: out * 2 + torch.flip(out, (0,)))
        dx, dgate, _ = ck.gated_recurrence_backward(d, gate, kept, g, state)
        pause()
        both = there(lambda: [dx * 3, dgate - 1])
        norm = ck.clip_gradients(both, 0.5)
        pause()
        logits = there(lambda: ((state + both[0][-1] + both[1][0] * norm) @ read).view(B, K, -1))
        scores, parents, tokens, _ = ck.beam_select(logits, scores)
        pause()
        again = there(lambda: (state + tokens.view(-1, 1) * 1e-4).view(B, K, -1))
        state = ck.reorder_states(again, parents).view(B * K, -1)
        pause()
    return state, scores, norm


def test_operands_from_another_stream():
    """In a row, with pauses, and captured with both streams: the same results."""
    g = torch.Generator().manual_seed(8)
    B, K, N, V, T = 2, 3, 500, 9000, 40
    x, gate = (torch.randn(T, B * K, N, generator=g).cuda() for _ in range(2))
    read, scores = (torch.randn(N, V, generator=g) * 0.1).cuda(), -torch.rand(B, K, generator=g).cuda()
    other = torch.cuda.Stream()
    want = handed_over(x, gate, read, scores, other, torch.cuda.synchronize)
    for _ in range(5):
        got = handed_over(x, gate, read, scores, other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = handed_over(x, gate, read, scores, other)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_from_several_threads():
    """Calls of several threads, each on a stream of its own."""
    import threading

    streams = [torch.cuda.Stream() for _ in range(4)]
    g = torch.Generator().manual_seed(9)
    sets = []
    for i in range(4):
        x, gate = (torch.randn(30 + i, 4, 100 + i, generator=g).cuda() for _ in range(2))
        sets.append((x, gate, (torch.randn(100 + i, 5000, generator=g) * 0.1).cuda(), -torch.rand(2, 2, generator=g).cuda()))
    want = [handed_over(*s, streams[0]) for s in sets]
    torch.cuda.synchronize()
    got, extra = [None] * 4, [torch.cuda.Stream() for _ in range(4)]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(5):
                got[i] = handed_over(*sets[i], extra[i])
            streams[i].synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for s, w in zip(got, want) for a, b in zip(s, w))
