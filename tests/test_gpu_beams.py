"""A step of beam search and the reordering of states against plain definitions."""
import numpy as np
import pytest
import torch

import sequence_oracle as so

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    return None if t is None else (t if t.dtype != torch.bfloat16 else t.float()).cpu().numpy()


def check(logits, scores, ended=None, end_token=None, beams=None):
    import sparse_graph_recurrent_gb300 as ck
    B, K, V = logits.shape
    want = so.beam(host(logits), host(scores), host(ended), -2 if end_token is None else end_token, beams or K)
    got = ck.beam_select(logits, scores, ended, end_token, beams)
    assert [t.dtype for t in got] == [torch.float32, torch.int64, torch.int64, torch.bool]
    for g, w in zip(got[1:], want[1:]):
        assert np.array_equal(host(g), w)
    some = want[2] >= 0
    assert np.array_equal(np.isfinite(host(got[0])), some)
    so.within(host(got[0])[some], want[0][some], so.beam_score_off(V))
    again = ck.beam_select(logits, scores, ended, end_token, beams)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


def make(B, K, V, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, K, V, generator=g) * 3).to(dtype).cuda(), (-torch.rand(B, K, generator=g) * 5).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V,beams", [
    (1, 1, 1, 1), (1, 1, 5, 3), (1, 4, 256, 4), (2, 3, 200, 5), (5, 8, 8191, 8), (1, 8, 8192, 8), (3, 2, 8193, 4),
    (2, 16, 50021, 16), (1, 64, 1000, 64), (1, 2, 131072, 64), (2, 5, 131075, 7), (40, 2, 33, 2), (1, 1, 40000, 1)])
def test_sizes(B, K, V, beams, dtype):
    check(*make(B, K, V, dtype, seed=V), beams=beams)


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_scores_go_to_the_lowest(dtype):
    for V in (7, 300, 8193, 20000):
        scores = torch.zeros(2, 4, device="cuda")
        got = check(torch.zeros(2, 4, V, dtype=dtype, device="cuda"), scores)
        assert (got[1] == 0).all() and torch.equal(got[2], torch.arange(4, device="cuda").expand(2, 4))
        # all beams alike, whole numbers among which there are many equals
        row = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(V)).to(dtype).cuda()
        check(row.expand(2, 4, V).contiguous(), scores)
        check(row.expand(2, 4, V), scores)
        check(row.expand(1, 64, V).contiguous(), torch.zeros(1, 64, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [300, 8192, 30001])
def test_sorted_logits(V, dtype):
    """All of the best in one thread's hands, at either end."""
    up = torch.linspace(-4, 4, V, device="cuda").to(dtype)
    for row in (up, up.flip(0)):
        check(torch.stack((row, row - 1, row + 1)).unsqueeze(0), torch.tensor([[0.0, -0.5, 0.25]], device="cuda"), beams=64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50, 9000])
def test_beams_that_have_ended(V, dtype):
    logits, scores = make(6, 5, V, dtype, seed=3)
    ended = torch.rand(6, 5, generator=torch.Generator().manual_seed(1)) < 0.5
    ended[0] = True
    ended[1] = False
    logits[2, :, 7] += 30  # the end token is likely
    got = check(logits, scores, ended.cuda(), 7)
    order = torch.sort(scores[0], descending=True)
    assert torch.equal(got[0][0], order.values) and torch.equal(got[1][0], order.indices) and got[3][0].all()
    check(logits, scores, None, 7)
    logits[:] = float("nan")  # a beam that has ended does not look at its logits
    check(logits, scores, ended.cuda(), 7)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_and_missing_candidates(dtype):
    inf, nan = float("inf"), float("nan")
    logits, scores = make(8, 4, 9001, dtype, seed=5)
    logits[0] = -inf                        # a sequence with nothing left
    logits[1, :, 3:] = -inf                 # fewer tokens than beams
    logits[2, 1:] = -inf                    # one beam left
    logits[3, 0, 17] = nan
    logits[3, 1, 9000] = inf
    logits[3, 2, :] = nan
    logits[4] = torch.finfo(dtype).min      # the type's lowest value is a logit like any other
    logits[4, 1, 8500:] = 0
    logits[7, :, :8999] = -inf
    logits[7, 1:] = -inf
    scores[5] = torch.tensor([0.0, -inf, -inf, -inf])  # a first step
    scores[6] = torch.tensor([nan, inf, -3.0, -1e30])
    for beams in (1, 4, 9):
        check(logits, scores, beams=beams)
    ended = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    ended[0, 2] = ended[6, 0] = ended[7, 3] = True
    check(logits, scores, ended, 11)


def test_strides():
    logits, scores = make(3, 4, 777, torch.float32)
    wide = torch.full((3, 4, 800), float("nan"), device="cuda")
    wide[..., 5:782] = logits
    want = check(logits, scores)
    for t in (wide[..., 5:782], logits.transpose(0, 1).contiguous().transpose(0, 1), logits.permute(2, 0, 1).contiguous().permute(1, 2, 0)):
        assert all(torch.equal(a, b) for a, b in zip(check(t, scores), want))
    half = wide[..., 5:782].half()
    odd = torch.empty(3 * 4 * 777 + 1, dtype=torch.float16, device="cuda")[1:].view(3, 4, 777).copy_(half)
    check(odd, scores.t().contiguous().t())


def test_nothing():
    import sparse_graph_recurrent_gb300 as ck
    got = ck.beam_select(torch.empty(0, 2, 5, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert all(t.shape == (0, 2) for t in got)


def test_selection_refusals():
    import sparse_graph_recurrent_gb300 as ck
    z, s = make(2, 3, 10, torch.float32)
    e = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    for bad in (lambda: ck.beam_select(z[0], s), lambda: ck.beam_select(z, s[:1]), lambda: ck.beam_select(z, s.half()),
                lambda: ck.beam_select(z.double(), s), lambda: ck.beam_select(z, s, e), lambda: ck.beam_select(z, s, e.int(), 3),
                lambda: ck.beam_select(z, s, e, 10), lambda: ck.beam_select(z, s, e, -1), lambda: ck.beam_select(z, s, beams=0),
                lambda: ck.beam_select(z, s, beams=65), lambda: ck.beam_select(z.cpu(), s), lambda: ck.beam_select(z, s.cpu()),
                lambda: ck.beam_select(z[..., :0], s), lambda: ck.beam_select(z.expand(2, 3, 10).repeat(1, 30, 1), s.repeat(1, 30)),
                lambda: ck.beam_select(z.clone().requires_grad_(), s)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()


# -- states ----------------------------------------------------------------------------------


def gathered(t, parents):
    B, beams = parents.shape
    out = torch.zeros(B, beams, *t.shape[2:], dtype=t.dtype)
    for b in range(B):
        for j in range(beams):
            p = int(parents[b, j])
            if 0 <= p < t.shape[1]:
                out[b, j] = t[b, p].cpu()
    return out


def some_states(B, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, K, 5000, generator=g).cuda(), torch.randint(0, 9, (B, K, 33), generator=g).cuda(),
            torch.randn(B, K, 77, generator=g).half().cuda(), torch.randn(B, K, 3, 5, generator=g).bfloat16().cuda(),
            (torch.rand(B, K, generator=g) < 0.5).cuda(), torch.randn(B, K, 1, generator=g).double().cuda(),
            torch.randint(0, 9, (B, K, 30011), generator=g).to(torch.uint8).cuda(), torch.empty(B, K, 0).cuda()]


@pytest.mark.parametrize("B,K,beams", [(1, 1, 1), (2, 4, 4), (3, 5, 8), (1, 64, 64), (7, 16, 2)])
def test_reorder(B, K, beams):
    import sparse_graph_recurrent_gb300 as ck
    states = some_states(B, K)
    parents = torch.randint(0, K, (B, beams), generator=torch.Generator().manual_seed(B)).cuda()
    want = [gathered(t, parents) for t in states]
    got = ck.reorder_states(states, parents)
    assert all(torch.equal(a.cpu(), b) and a.dtype == b.dtype and a.shape == b.shape for a, b in zip(got, want))
    assert torch.equal(ck.reorder_states(states[0], parents).cpu(), want[0])
    out = [torch.full_like(t, 1) for t in got]
    assert all(a is b for a, b in zip(ck.reorder_states(states, parents, out=out), out))
    assert all(torch.equal(a.cpu(), b) for a, b in zip(out, want))
    if beams == K:
        mixed = [t if i % 2 else torch.empty_like(t) for i, t in enumerate(states)]
        ck.reorder_states(states, parents, out=mixed)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(mixed, want))


def test_parents_that_are_no_beams_give_zeros():
    import sparse_graph_recurrent_gb300 as ck
    states = some_states(3, 4)
    parents = torch.tensor([[0, -1, 4, 3], [2 ** 40, -2 ** 63, 1, 1], [3, 2, 1, 0]], device="cuda")
    want = [gathered(t, parents) for t in states]
    assert all(torch.equal(a.cpu(), b) for a, b in zip(ck.reorder_states(states, parents), want))
    ck.reorder_states(states, parents, out=states)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(states, want))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.float32, torch.float64])
def test_rows_of_any_length_and_place(dtype):
    import sparse_graph_recurrent_gb300 as ck
    for n in (1, 3, 15, 16, 17, 1023, 8191, 8193, 20001):
        for a, b in ((0, 0), (1, 0), (0, 1), (3, 2)):
            whole = torch.randint(0, 100, (2, 3, n + 9)).to(dtype).cuda()
            to = torch.full((2, 3, n + 5), 7, dtype=dtype, device="cuda")
            parents = torch.tensor([[2, 0, 0], [1, 1, 2]], device="cuda")
            part = whole[..., a:a + n]
            ck.reorder_states(part, parents, out=to[..., b:b + n])
            want = gathered(part, parents)
            assert torch.equal(to[..., b:b + n].cpu(), want)
            assert (to[..., :b] == 7).all() and (to[..., b + n:] == 7).all()
            assert torch.equal(ck.reorder_states(part, parents).cpu(), want)
            keep = whole.clone()
            ck.reorder_states([part], parents, out=[part])
            assert torch.equal(part.cpu(), want)
            assert torch.equal(whole[..., :a], keep[..., :a]) and torch.equal(whole[..., a + n:], keep[..., a + n:])


def test_orders_of_axes_and_columns_of_one_array():
    import sparse_graph_recurrent_gb300 as ck
    parents = torch.tensor([[1, 1, 0], [2, 0, 2]], device="cuda")
    t = torch.randn(3, 2, 40, device="cuda").transpose(0, 1)  # beams outermost
    assert torch.equal(ck.reorder_states(t, parents).cpu(), gathered(t, parents))
    want = gathered(t, parents)
    ck.reorder_states(t, parents, out=t)
    assert torch.equal(t.cpu(), want)
    both = torch.randn(2, 3, 100, device="cuda")
    parts = [both[..., :30], both[..., 30:100]]
    want = [gathered(p, parents) for p in parts]
    ck.reorder_states(parts, parents, out=parts)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(parts, want))
    u = torch.randn(2, 3, 4, 5, device="cuda").transpose(2, 3)
    assert torch.equal(ck.reorder_states(u, parents).cpu(), gathered(u, parents))
    one = torch.randn(1, 1, 40, device="cuda").expand(2, 3, 40)
    assert torch.equal(ck.reorder_states(one, parents).cpu(), gathered(one, parents))


def test_many_states():
    import sparse_graph_recurrent_gb300 as ck
    states = [torch.randn(2, 3, 5 + i, device="cuda") for i in range(70)]
    parents = torch.tensor([[1, 1, 0], [2, 0, 2]], device="cuda")
    want = [gathered(t, parents) for t in states]
    assert all(torch.equal(a.cpu(), b) for a, b in zip(ck.reorder_states(states, parents), want))
    ck.reorder_states(states, parents, out=states)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(states, want))
    assert ck.reorder_states([], parents) == []


def test_reorder_refusals():
    import sparse_graph_recurrent_gb300 as ck
    t = torch.randn(2, 3, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    for bad in (lambda: ck.reorder_states(t, p.int()), lambda: ck.reorder_states(t, p[0]), lambda: ck.reorder_states(t.cpu(), p),
                lambda: ck.reorder_states([t, t[:, :2]], p), lambda: ck.reorder_states(t[0], p), lambda: ck.reorder_states(t, p.cpu()),
                lambda: ck.reorder_states(t, p, out=t[:, :2]), lambda: ck.reorder_states(t, p, out=t.half()),
                lambda: ck.reorder_states([t], p, out=[]), lambda: ck.reorder_states(t, p[:, :2], out=t[:, :2]),
                lambda: ck.reorder_states([t, t], p, out=[t, t]), lambda: ck.reorder_states(t[..., :7], p, out=t[..., 1:]),
                lambda: ck.reorder_states(t, p, out=torch.empty(2, 3, 8, device="cuda").transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: ck.reorder_states(t, p, out=torch.empty(1, 1, 8, device="cuda").expand(2, 3, 8)),
                lambda: ck.reorder_states(t.clone().requires_grad_(), p)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()


# -- together --------------------------------------------------------------------------------


def test_captured_and_replayed():
    import sparse_graph_recurrent_gb300 as ck
    logits, scores = make(2, 4, 20001, torch.bfloat16, seed=1)
    more, other = make(2, 4, 20001, torch.bfloat16, seed=2)
    state = torch.randn(2, 4, 501, device="cuda")
    ended = torch.zeros(2, 4, dtype=torch.bool, device="cuda")

    def step():
        s, p, t, e = ck.beam_select(logits, scores, ended, 5)
        return s, p, t, e, ck.reorder_states(state, p)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for a, b in ((logits, more), (scores, other)):
        a.copy_(b)
    ended[1, 2] = True
    want = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_search_finds_what_trying_all_sequences_finds():
    """Three steps of a small gated model whose next logits depend on its state, with as
    many beams as there are prefixes: the best sequences of all."""
    import itertools

    import sparse_graph_recurrent_gb300 as ck
    V, N, steps, beams = 4, 6, 3, 16
    g = torch.Generator().manual_seed(4)
    embed, gates, read = (torch.randn(V, N, generator=g).cuda() for _ in range(3))
    state0 = torch.randn(1, N, generator=g).cuda()

    def advance(tokens, state):
        return ck.gated_recurrence(embed[tokens].unsqueeze(0), gates[tokens].unsqueeze(0), state)[1]
    scores = torch.full((1, beams), -float("inf"), device="cuda")
    scores[0, 0] = 0
    state = state0.expand(beams, N).contiguous().view(1, beams, N)
    text = torch.zeros(1, beams, steps, dtype=torch.int64, device="cuda")
    for i in range(steps):
        logits = (state.view(beams, N) @ read.t()).view(1, beams, V)
        scores, parents, tokens, _ = ck.beam_select(logits, scores)
        state, text = ck.reorder_states([state, text], parents)
        text[..., i] = tokens
        state = advance(tokens.view(-1), state.view(beams, N)).view(1, beams, N)
    e, f, r, s0 = (t.double().cpu().numpy() for t in (embed, gates, read, state0[0]))
    every = []
    for seq in itertools.product(range(V), repeat=steps):
        s, total = s0, 0.0
        for v in seq:
            z = r @ s
            total += z[v] - np.log(np.exp(z).sum())
            leak = 1 / (1 + np.exp(-f[v]))
            s = (1 - leak) * s + leak * e[v]
        every.append((-total, seq))
    every.sort()
    assert [tuple(t) for t in text[0].tolist()] == [seq for _, seq in every[:beams]]
    assert np.abs(scores[0].cpu().numpy() + np.array([v for v, _ in every[:beams]])).max() < 1e-4
