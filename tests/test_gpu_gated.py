"""The gated recurrence against its definition in 64 bits, both forms, both directions."""
import numpy as np
import pytest
import torch

import sequence_oracle as so

pytestmark = pytest.mark.gpu

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(T, B, N, dtype, form, seed=0, lengths=False, state0=True):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    dt = TYPES[dtype]
    x = rand(T, B, N).to(dt).cuda()
    gate = (rand(T, B, N) * 2 if form == "leak" else torch.sigmoid(rand(T, B, N) * 2 + 2)).to(dt).cuda()
    d = dict(x=x, gate=gate, state0=rand(B, N).cuda() if state0 else None, lengths=None,
             d_out=rand(T, B, N).to(dt).cuda(), d_state=rand(B, N).cuda())
    if lengths:
        n = torch.randint(0, T + 1, (B,), generator=g)
        n[0] = T
        n[-1] = 0
        d["lengths"] = n.cuda()
    return d


def check(d, form, dtype):
    import sparse_graph_recurrent_gb300 as ck
    want, off = so.gated(host(d["x"]), host(d["gate"]), host(d["state0"]),
                         None if d["lengths"] is None else d["lengths"].cpu().numpy(), form, host(d["d_out"]),
                         host(d["d_state"]))
    out, state = ck.gated_recurrence(d["x"], d["gate"], d["state0"], d["lengths"], form)
    o2, s2, kept = ck.gated_recurrence_forward(d["x"], d["gate"], d["state0"], d["lengths"], form)
    assert torch.equal(out, o2) and torch.equal(state, s2)
    assert out.dtype == d["x"].dtype and state.dtype == torch.float32
    dx, dgate, dstate0 = ck.gated_recurrence_backward(d["x"], d["gate"], kept, d["d_out"], d["d_state"], d["lengths"], form)
    for name, t, dt in (("out", out, dtype), ("state", state, "float32"), ("dx", dx, dtype), ("dgate", dgate, dtype),
                        ("dstate0", dstate0, "float32")):
        so.within(host(t), want[name], off[name], dt)
    again = ck.gated_recurrence_backward(d["x"], d["gate"], kept, d["d_out"], d["d_state"], d["lengths"], form)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgate, dstate0)))


SIZES = [(1, 1, 1), (1, 8, 256), (2, 3, 5), (15, 1, 2), (16, 2, 7), (17, 2, 64), (33, 5, 13), (128, 1, 33), (129, 3, 6),
         (500, 2, 1), (1025, 1, 66), (4999, 1, 10), (6000, 3, 35)]


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,B,N", SIZES)
def test_both_directions(T, B, N, dtype, form):
    check(inputs(T, B, N, dtype, form, seed=T + N), form, dtype)


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,B,N", [(1, 4, 3), (17, 5, 9), (64, 7, 11), (300, 3, 8), (5000, 2, 5)])
def test_lengths(T, B, N, dtype, form):
    check(inputs(T, B, N, dtype, form, seed=T, lengths=True), form, dtype)
    check(inputs(T, B, N, dtype, form, seed=T, lengths=True, state0=False), form, dtype)


def test_lengths_out_of_range_are_clamped():
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(20, 3, 4, "float32", "leak")
    a = ck.gated_recurrence(d["x"], d["gate"], d["state0"], torch.tensor([-3, 2 ** 40, 7], device="cuda"))
    b = ck.gated_recurrence(d["x"], d["gate"], d["state0"], torch.tensor([0, 20, 7], device="cuda"))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [40, 4100])
def test_what_lies_behind_a_sequence_is_not_looked_at(T, dtype):
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(T, 3, 5, dtype, "leak", lengths=True)
    n = d["lengths"].tolist()
    clean = {k: None if v is None else v.clone() for k, v in d.items()}
    for b in range(3):
        d["x"][n[b]:, b] = float("nan")
        d["gate"][n[b]:, b] = float("inf")
        d["d_out"][n[b]:, b] = float("nan")
    for form in ("leak", "decay"):
        res = []
        for v in (d, clean):
            out, state, kept = ck.gated_recurrence_forward(v["x"], v["gate"], v["state0"], v["lengths"], form)
            res.append((out, state, *ck.gated_recurrence_backward(v["x"], v["gate"], kept, v["d_out"], v["d_state"], v["lengths"], form)))
        # bit for bit: gates beyond 1 let a decay's states leave 32 bits, to infinities and NaN
        bits = {2: torch.int16, 4: torch.int32}
        assert all(torch.equal(*(t.view(bits[t.element_size()]) for t in pair)) for pair in zip(*res))


@pytest.mark.parametrize("form", ["leak", "decay"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("make", ["sequences_first", "wider_rows", "odd_start", "swapped", "every_second", "one_sequence"])
def test_strides(make, dtype, form):
    T, B, N = 150, 4, 6

    def lay(t):
        if make == "sequences_first":
            return t.transpose(0, 1).contiguous().transpose(0, 1)
        if make == "wider_rows":
            w = torch.full((T, B, N + 3), float("nan"), dtype=t.dtype, device="cuda")
            w[..., 2:2 + N] = t
            return w[..., 2:2 + N]
        if make == "odd_start":
            w = torch.empty(T * B * N + 1, dtype=t.dtype, device="cuda")[1:].view(T, B, N)
            return w.copy_(t)
        if make == "swapped":
            return t.permute(2, 1, 0).contiguous().permute(2, 1, 0)
        if make == "every_second":
            w = torch.empty(T, 2 * B, N, dtype=t.dtype, device="cuda")[:, ::2]
            return w.copy_(t)
        return t
    d = inputs(T, 1 if make == "one_sequence" else B, N, dtype, form, lengths=True)
    for name in ("x", "gate", "d_out"):
        d[name] = lay(d[name])
    check(d, form, dtype)
    plain = inputs(T, 1 if make == "one_sequence" else B, N, dtype, form, lengths=True)
    plain["x"] = d["x"]  # operands of different layouts
    check(plain, form, dtype)


@pytest.mark.parametrize("shape", [(1, 1, 6), (70, 1, 6), (1, 4, 6), (70, 4, 1), (70, 1, 1), (6,)])
def test_a_gate_that_expands_gets_the_summed_gradient(shape):
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(70, 4, 6, "float32", "leak")
    gate = torch.randn(shape, device="cuda", requires_grad=True)
    full = gate.detach().expand(70, 4, 6).contiguous().requires_grad_()
    for g in (gate, full):
        out, state = ck.gated_recurrence(d["x"], g, d["state0"])
        torch.autograd.backward((out, state), (d["d_out"], d["d_state"]))
    want = host(full.grad)
    axes = tuple(i - len(shape) + 3 for i, n in enumerate(shape) if n == 1)
    axes += tuple(range(3 - len(shape)))
    s, size = want.sum(axis=axes, keepdims=True).reshape(shape), np.abs(want).sum(axis=axes, keepdims=True).reshape(shape)
    # sums of at most 1,680 numbers of 32 bits, in any order
    assert (np.abs(host(gate.grad) - s) <= 1680 * so.U32 * size).all()


def test_autograd_gives_the_backward():
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(37, 3, 10, "bfloat16", "decay", lengths=True)
    leaves = [d[k].detach().requires_grad_() for k in ("x", "gate", "state0")]
    out, state = ck.gated_recurrence(*leaves, d["lengths"], "decay")
    _, _, kept = ck.gated_recurrence_forward(*leaves, d["lengths"], "decay")
    for d_out, d_state in ((d["d_out"], d["d_state"]), (None, d["d_state"]), (d["d_out"], None)):
        some = [(o, g) for o, g in ((out, d_out), (state, d_state)) if g is not None]
        got = torch.autograd.grad([o for o, _ in some], leaves, [g for _, g in some], retain_graph=True)
        want = ck.gated_recurrence_backward(d["x"], d["gate"], kept, d_out, d_state, d["lengths"], "decay")
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    only = torch.autograd.grad(out, leaves[1], d["d_out"], retain_graph=True)[0]
    assert torch.equal(only, ck.gated_recurrence_backward(d["x"], d["gate"], kept, d["d_out"], None, d["lengths"], "decay")[1])
    with pytest.raises(RuntimeError):
        g = torch.autograd.grad(out, leaves[0], d["d_out"], create_graph=True)[0]
        torch.autograd.grad(g.float().sum(), leaves[0])


def test_steps_one_by_one_are_the_whole():
    """A sequence answered step by step, the state passed on, agrees with its window."""
    import sparse_graph_recurrent_gb300 as ck
    d = inputs(21, 2, 50, "float16", "leak")
    want, off = so.gated(host(d["x"]), host(d["gate"]), host(d["state0"]), None, "leak")
    state, outs = d["state0"], []
    for t in range(21):
        out, state = ck.gated_recurrence(d["x"][t:t + 1], d["gate"][t:t + 1], state)
        outs.append(out)
    so.within(host(torch.cat(outs)), want["out"], off["out"], "float16")
    so.within(host(state), want["state"], off["state"])


def test_no_steps_and_no_nodes():
    import sparse_graph_recurrent_gb300 as ck
    s = torch.randn(3, 4, device="cuda")
    x = torch.empty(0, 3, 4, device="cuda")
    out, state, kept = ck.gated_recurrence_forward(x, x, s)
    assert out.shape == (0, 3, 4) and torch.equal(state, s)
    assert not ck.gated_recurrence(x, x)[1].any()
    dx, dgate, ds = ck.gated_recurrence_backward(x, x, kept, x, s)
    assert dx.shape == dgate.shape == x.shape and torch.equal(ds, s)
    x = torch.empty(5, 0, 4, device="cuda")
    out, state = ck.gated_recurrence(x, x)
    assert out.shape == (5, 0, 4) and state.shape == (0, 4)


def test_values_that_are_not_finite_stay_in_their_place():
    """They reach later steps of their own node alone."""
    import sparse_graph_recurrent_gb300 as ck
    for T in (60, 5000):
        d = inputs(T, 2, 6, "float32", "leak")
        clean = ck.gated_recurrence(d["x"], d["gate"], d["state0"])[0]
        d["x"][T // 2, 1, 3] = float("nan")
        d["x"][T // 3, 0, 1] = float("inf")
        out = ck.gated_recurrence(d["x"], d["gate"], d["state0"])[0]
        touched = torch.zeros_like(out, dtype=torch.bool)
        touched[T // 2:, 1, 3] = True
        touched[T // 3:, 0, 1] = True
        assert torch.equal(out[~touched], clean[~touched])
        assert out[T // 2:, 1, 3].isnan().all() and (out[T // 3:, 0, 1] == float("inf")).all()


def test_extreme_gates():
    """A leak of 0 or 1 to the last bit, and gates that are infinite."""
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(40, 1, 4, device="cuda")
    gate = torch.tensor([1e4, -1e4, float("inf"), -float("inf")], device="cuda").expand(40, 1, 4)
    s = torch.randn(1, 4, device="cuda")
    out, state = ck.gated_recurrence(x, gate, s)
    assert torch.equal(out[..., 0::2], x[..., 0::2]) and torch.equal(out[..., 1::2], s[None, :, 1::2].expand(40, 1, 2))


def test_captured_and_replayed():
    import sparse_graph_recurrent_gb300 as ck
    d, e = (inputs(3000, 2, 9, "float32", "leak", seed=i, lengths=True) for i in (1, 2))

    def step(d):
        out, state, kept = ck.gated_recurrence_forward(d["x"], d["gate"], d["state0"], d["lengths"])
        return (out, state, *ck.gated_recurrence_backward(d["x"], d["gate"], kept, d["d_out"], d["d_state"], d["lengths"]))
    want = [step(v) for v in (d, e)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    for k in ("x", "gate", "state0", "lengths", "d_out", "d_state"):
        d[k].copy_(e[k])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


def test_two_streams_at_once():
    import sparse_graph_recurrent_gb300 as ck
    ds = [inputs(4000, 1, 30 + i, "float32", "decay", seed=i) for i in range(2)]
    want = [ck.gated_recurrence(d["x"], d["gate"], d["state0"], None, "decay") for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(10):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(ck.gated_recurrence(d["x"], d["gate"], d["state0"], None, "decay"))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_many_nodes():
    """More nodes than one wave of the device holds, and rows that pairs cannot take."""
    for N, dtype in ((60001, "float32"), (200000, "float16")):
        check(inputs(19, 1, N, dtype, "leak"), "leak", dtype)


def test_refusals():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(5, 2, 4, device="cuda")
    s, n = torch.zeros(2, 4, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    good = dict(x=x, gate=x, state0=s, lengths=n, form="leak")
    ck.gated_recurrence(**good)
    for bad in (dict(x=x[0]), dict(gate=x.half()), dict(gate=x.cpu()), dict(x=x.double(), gate=x.double()), dict(state0=s.half()),
                dict(state0=s[:1]), dict(lengths=n.int()), dict(lengths=n[:1]), dict(lengths=n.cpu()), dict(form="no"),
                dict(x=x.cpu())):
        with pytest.raises((ValueError, RuntimeError)):
            ck.gated_recurrence(**{**good, **bad})
    _, _, kept = ck.gated_recurrence_forward(x, x)
    for bad in (dict(kept=kept[:-1]), dict(d_out=x[:4]), dict(d_out=x.half()), dict(d_state=s.half()), dict(kept=kept.half())):
        with pytest.raises(ValueError):
            ck.gated_recurrence_backward(**{**dict(x=x, gate=x, kept=kept, d_out=x, d_state=s), **bad})
