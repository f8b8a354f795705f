"""The global gradient norm and clipping against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import sequence_oracle as so
import workloads
from gpu_helpers import make_graph, to_dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "float32", BF16: "bfloat16", F16: "float16"}

# Of a sum of squares, in half steps: the product, 32 additions of a thread in a chunk, one
# for each chunk of a CTA (no more than 20 here); then 64 bits.  The root halves that and is rounded.
NORM_OFF = ((1 + 32 + 20) / 2 + 1) * so.U32
FACTOR_OFF = NORM_OFF + 2 * so.U32


def host(t):
    return t.detach().double().cpu().numpy()


def make(sizes, types, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(t).cuda() for n, t in zip(sizes, types)]


def check(grads, max_norm, out=None):
    import sparse_graph_recurrent_gb300 as ck
    want = [host(g) for g in grads]
    norm, factor = so.clip(want, max_norm)
    alone = ck.grad_norm(grads)
    got = ck.clip_gradients(grads, max_norm, out=out)
    assert alone.dtype == got.dtype == F32 and alone.shape == got.shape == ()
    assert torch.equal(alone, got)
    assert abs(float(got) - norm) <= NORM_OFF * norm + 2.0 ** -149
    for t, w in zip(grads if out is None else out, want):
        so.within(host(t), w * factor, np.abs(w * factor) * FACTOR_OFF, NAMES[t.dtype])
    if out is not None:
        assert all(np.array_equal(host(g), w) for g, w in zip(grads, want))


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9])
@pytest.mark.parametrize("sizes,types", [
    ([1], [F32]), ([7], [BF16]), ([4096, 256, 256], [F32] * 3), ([5, 0, 70001], [F16, F32, BF16]),
    ([4095, 4096, 4097, 8191, 8193], [F32, BF16, F16, F16, F32]), ([3_000_001, 17], [F32, F32]), ([5_000_003], [BF16]),
])
def test_sizes_and_types(sizes, types, max_norm):
    check(make(sizes, types), max_norm)
    grads = make(sizes, types)
    check(grads, max_norm, [torch.empty_like(g) for g in grads])


@pytest.mark.parametrize("count", [32, 33, 999, 1000, 1001, 2503])
def test_many_tensors(count):
    rng = np.random.default_rng(count)
    sizes = [int(n) for n in np.exp(rng.uniform(0, 9, count))]
    types = [(F32, BF16, F16)[i % 3] for i in range(count)]
    check(make(sizes, types), 0.7)
    grads = make(sizes, types)
    check(grads, 0.7, [torch.empty_like(g) for g in grads])


@pytest.mark.parametrize("a,b", [(0, 0), (1, 0), (0, 1), (1, 1), (3, 5)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_any_alignment(dtype, a, b):
    for n in (1, 2, 9, 4096, 20011):
        big = make([n + 16], [dtype])[0]
        to = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
        check([big[a:a + n]], 0.1, [to[b:b + n]])
        assert (to[:b] == 7).all() and (to[b + n:] == 7).all()
        before = big.clone()
        check([big[a:a + n]], 0.1)
        assert torch.equal(big[:a], before[:a]) and torch.equal(big[a + n:], before[a + n:])


def test_strides_and_orders():
    import sparse_graph_recurrent_gb300 as ck
    base = torch.randn(60, 50, 4, device="cuda")
    for view in (lambda t: t.permute(2, 0, 1), lambda t: t[:, ::2], lambda t: t[..., 1], lambda t: t[3:4, :, :2]):
        for out in (False, True):
            t = base.clone()
            keep = t.clone()
            g = view(t)
            want = host(g)
            norm, factor = so.clip([want], 1.5)
            o = view(torch.zeros_like(t)) if out else None
            got = ck.clip_gradients([g], 1.5, out=None if o is None else [o])
            assert abs(float(got) - norm) <= NORM_OFF * norm
            so.within(host(o if out else g), want * factor, np.abs(want * factor) * FACTOR_OFF)
            if not out:  # what lies between is as it was
                view(t).copy_(view(keep))
            assert torch.equal(t, keep)
    # one dense and one not, of the same elements
    t = base.clone()
    o = torch.empty(4, 60, 50, device="cuda")
    ck.clip_gradients(t.permute(2, 0, 1), 1.5, out=o)
    norm, factor = so.clip([host(t)], 1.5)
    so.within(host(o), host(t.permute(2, 0, 1)) * factor, np.abs(host(t.permute(2, 0, 1))) * factor * FACTOR_OFF)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e25, 1e19, 1e-12, 1e-25, 1e-33])
def test_squares_that_leave_32_bits(scale, dtype):
    """The norm is the scale's multiple all the same; alone and beside ordinary numbers."""
    import sparse_graph_recurrent_gb300 as ck
    g = make([3000, 77], [dtype, F32], scale)
    want = [host(t) for t in g]
    norm, _ = so.clip(want, 1.0)
    assert abs(float(ck.grad_norm(g)) - norm) <= NORM_OFF * norm
    g.append(torch.ones(5, device="cuda"))
    norm, factor = so.clip([host(t) for t in g], 1.0)
    assert abs(float(ck.clip_gradients(g, 1.0)) - norm) <= NORM_OFF * norm
    for t, w in zip(g, want):
        so.within(host(t), w * factor, np.abs(w * factor) * FACTOR_OFF, NAMES[t.dtype])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_what_is_not_finite(dtype):
    import sparse_graph_recurrent_gb300 as ck
    for bad in (float("inf"), -float("inf"), float("nan")):
        a, b = make([10000, 5], [dtype, F32])
        a[7000] = bad
        was = host(a)
        norm = float(ck.clip_gradients([a, b], 1.0))
        if bad != bad:
            assert norm != norm and a.isnan().all() and b.isnan().all()
        else:
            assert norm == float("inf")
            assert host(a)[7000] != host(a)[7000] and not b.any()  # inf times 0, and 0
            assert not np.delete(host(a), 7000).any() and np.isinf(was[7000])


def test_nothing_to_clip():
    import sparse_graph_recurrent_gb300 as ck
    assert float(ck.grad_norm([])) == 0 and float(ck.clip_gradients([], 1.0)) == 0
    assert float(ck.clip_gradients([None, torch.empty(0, device="cuda")], 1.0)) == 0
    z = torch.zeros(1000, device="cuda")
    assert float(ck.clip_gradients([z, None], 1.0)) == 0 and not z.any()
    g = make([100], [F32])[0]
    assert abs(float(ck.clip_gradients(g, 0.5)) - np.linalg.norm(host(make([100], [F32])[0]))) < 1e-4


def test_one_device_tensor_counts_twice_where_only_read():
    import sparse_graph_recurrent_gb300 as ck
    g = make([1000], [F32])[0]
    assert abs(float(ck.grad_norm([g, g])) - np.sqrt(2) * np.linalg.norm(host(g))) <= 4 * NORM_OFF * 50


def test_refusals():
    import sparse_graph_recurrent_gb300 as ck
    g = make([1000], [F32])[0]
    for bad in (lambda: ck.clip_gradients([g, g], 1.0), lambda: ck.clip_gradients([g, g[10:20]], 1.0),
                lambda: ck.clip_gradients([g], 1.0, out=[g.half()]), lambda: ck.clip_gradients([g], 1.0, out=[]),
                lambda: ck.clip_gradients([g[:500]], 1.0, out=[g[1:501]]), lambda: ck.clip_gradients([g], float("nan")),
                lambda: ck.clip_gradients([g], -1.0), lambda: ck.clip_gradients([g.cpu()], 1.0),
                lambda: ck.clip_gradients([g.double()], 1.0), lambda: ck.grad_norm([g.long()]),
                lambda: ck.clip_gradients([g[:10], g[10:20]], 1.0, out=[g[100:110], g[105:115]]),
                lambda: ck.clip_gradients([g.clone().requires_grad_()], 1.0),
                lambda: ck.clip_gradients([g], 1.0, out=[g[:10]])):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    ck.clip_gradients([g[:10], g[10:20]], 1.0, out=[g[20:30], g[30:40]])  # side by side is fine


def test_a_clipped_tensor_is_written():
    import sparse_graph_recurrent_gb300 as ck
    g = make([100], [F32])[0]
    v = g._version
    ck.clip_gradients([g], 0.1)
    assert g._version > v


def test_captured_and_replayed_and_repeated():
    import sparse_graph_recurrent_gb300 as ck
    grads = make([50_000, 1234, 999_999], [F32, BF16, F32])
    out = [torch.empty_like(g) for g in grads]
    ck.clip_gradients(grads, 1.0, out=out)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two that share nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = ck.clip_gradients(grads, 1.0, out=out)
        graphs.append((graph, norm))
    other = make([50_000, 1234, 999_999], [F32, BF16, F32], scale=3.0, seed=9)
    for g, o in zip(grads, other):
        g.copy_(o)
    want = ck.clip_gradients(other, 1.0)
    for graph, norm in graphs:
        for o in out:
            o.zero_()
        graph.replay()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, other))


def test_streams_at_once():
    import sparse_graph_recurrent_gb300 as ck
    sets = [make([300_000 + i, 70], [F32, BF16], seed=i) for i in range(3)]
    want = [[torch.empty_like(g) for g in s] for s in sets]
    norms = [ck.clip_gradients(s, 1.0, out=w) for s, w in zip(sets, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [[torch.empty_like(g) for g in s] for s in sets]
        torch.cuda.synchronize()
        n = []
        for s, g, st in zip(sets, got, streams):
            with torch.cuda.stream(st):
                n.append(ck.clip_gradients(s, 1.0, out=g))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(n, norms))
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


@pytest.mark.parametrize("optimizer", ["sgd", "adam"])
def test_a_captured_training_step_clips(optimizer):
    """TrainStep(max_norm=) is the same calls made one after another."""
    import sparse_graph_recurrent_gb300 as pkg
    from sparse_graph_recurrent_gb300 import _ck
    c = workloads.small(501, 200, 8000, 10, 24, 3, 2)
    g = make_graph(c)
    M, T, B = c["M"], c["drives"].shape[0], c["state0"].shape[0]
    fixed = {k: to_dev(c[k]) for k in ("drives", "state0", "dout")}
    eager, cap = ({k: to_dev(c[k]) for k in ("w", "leak", "bias")} for _ in range(2))
    moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in eager.items()}
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = 1e-3
    step = pkg.TrainStep(g, cap["w"], cap["leak"], cap["bias"], fixed["drives"], fixed["state0"], fixed["dout"], M, lr,
                         optimizer=optimizer, max_norm=0.25)
    for _ in range(3):
        step()
        _, saved, scratch = pkg.forward(g, eager["w"], eager["leak"], eager["bias"], fixed["drives"], fixed["state0"], M)
        grads = pkg.backward(g, eager["w"], eager["leak"], B, T, M, saved, fixed["dout"], scratch)[:3]
        norm = pkg.clip_gradients(grads, 0.25)
        if optimizer == "sgd":
            for k, d in zip(("w", "leak", "bias"), grads):
                _ck.ck_sgd_update(eager[k], d, lr)
        else:
            _ck.ck_step_advance(count)
            for k, d in zip(("w", "leak", "bias"), grads):
                _ck.ck_adam_update(eager[k], d, *moments[k], count, lr)
        assert float(norm) > 0.25 and torch.equal(step.norm, norm.view(1))
    for k in cap:
        assert torch.equal(cap[k], eager[k]), k
