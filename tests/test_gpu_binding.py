"""The compiled module ck_binding and the Python form of the same calls agree, and
what the module does not take the Python form does or refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Nothing:
    """A module that leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture
def both(monkeypatch):
    from sparse_graph_recurrent_gb300 import _ck
    native = _ck.native()

    def run(call):
        monkeypatch.setattr(_ck, "_native", native)
        a = call()
        monkeypatch.setattr(_ck, "_native", Nothing())
        b = call()
        monkeypatch.setattr(_ck, "_native", native)
        return a, b
    return run


def same(a, b):
    if isinstance(a, tuple):
        assert len(a) == len(b)
        return all(same(x, y) for x, y in zip(a, b))
    return a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and torch.equal(a, b)


def test_dropout_both_ways(both):
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(4, 6, 130, device="cuda")
    step = torch.tensor([3], device="cuda")
    for v in (x, x[..., :121], x.transpose(0, 1), x.permute(2, 0, 1)[::2], x[:1].expand(4, 6, 130), x.half(), x[0, 0]):
        for locked in (False, True) if v.dim() > 1 else (False,):
            for s in (0, -1, 2 ** 64 - 1, step):
                assert same(*both(lambda: ck.dropout(v, 0.4, 2 ** 63 + 1, s, locked=locked)))
    assert same(*both(lambda: ck.dropout(x, 1, 5)))
    assert same(*both(lambda: ck.dropout_backward(x, 0.5, 5, 6)))


def test_int4_both_ways(both):
    import sparse_graph_recurrent_gb300 as ck
    w = torch.randn(70, 333, device="cuda")
    for symmetric in (True, False):
        q, s, z = ck.int4_quantize(w, 32, symmetric, scale_dtype=torch.bfloat16)
        for M in (1, 5):
            x = torch.randn(M, 333, device="cuda")
            for bias in (None, torch.randn(70, device="cuda")):
                assert same(*both(lambda: ck.int4_matvec(x, q, s, z, bias, 32)))
            out = torch.empty(M, 80, device="cuda")[:, :70]
            assert same(*both(lambda: ck.int4_matvec(x, q, s, z, group_size=32, out=out).clone()))
    assert same(*both(lambda: ck.int4_matvec(w[0], q, s, z, group_size=32)))
    assert same(*both(lambda: ck.int4_matvec(w[:1], q[:1], s[:1], z[:1], group_size=32)))


def test_controls_both_ways(both):
    import sparse_graph_recurrent_gb300 as ck
    B, V = 3, 9001
    x = torch.randn(B, V, device="cuda")
    h = torch.randint(0, V, (B, 50), device="cuda")
    n = torch.tensor([50, 3, 0], device="cuda")
    rows = torch.rand(B, device="cuda") + 0.5
    step = torch.tensor([9], device="cuda")
    for kw in ({}, dict(history=h), dict(history=h.int(), history_len=n.int()), dict(temperature=0.7), dict(temperature=0),
               dict(history=h, history_len=n, prompt_len=n // 2, repetition=1.2, frequency=rows, presence=rows,
                    temperature=rows, bias=torch.randn(V, device="cuda"),
                    mask=torch.full((B, -(-V // 32)), -2, dtype=torch.int32, device="cuda"))):
        assert same(*both(lambda: ck.control_logits(x, **kw)))
        for seed in (None, 5):
            for s in (2, step):
                assert same(*both(lambda: ck.pick_tokens(x, **kw, seed=seed, step=s)))
                assert same(*both(lambda: ck.pick_tokens(x, **kw, seed=seed, step=s, return_logits=True)))


def test_what_the_module_leaves():
    from sparse_graph_recurrent_gb300 import _ck
    n = _ck.native()
    x = torch.randn(2, 64, device="cuda", requires_grad=True)
    assert n.dropout(x, 0.5, 1, 0, False) is None
    assert n.dropout(x.detach().double(), 0.5, 1, 0, False) is None
    assert n.dropout(x.detach().cpu(), 0.5, 1, 0, False) is None
    assert n.dropout(x.detach(), 0.5, "1", 0, False) is None
    assert n.dropout(None, 0.5, 1, 0, False) is None
    with torch.no_grad():
        assert n.dropout(x, 0.5, 1, 0, False) is not None
    with pytest.raises(_ck.CKError) as e:
        n.dropout(x.detach(), 1.5, 1, 0, False)
    assert e.value.name == "CK_ERR_INVALID_ARG"


def test_writing_into_a_tensor_raises_its_version(both):
    """autograd finds a saved tensor that `out` has changed since."""
    import sparse_graph_recurrent_gb300 as ck
    q, s, _ = ck.int4_quantize(torch.randn(64, 64, device="cuda"), 32)
    x = torch.randn(2, 64, device="cuda")
    for call in (lambda o: ck.int4_matvec(x, q, s, group_size=32, out=o), lambda o: ck.control_logits(x, out=o),
                 lambda o: ck.pick_tokens(x, out=o), lambda o: ck.control_logits(o, out=o)):
        def run():
            a = torch.randn(2, 64, device="cuda", requires_grad=True)
            saved = torch.randn(2, 64, device="cuda")
            y = (a * saved).sum()
            at = saved._version
            call(saved)
            assert saved._version == at + 1
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
        both(run)


def test_numpy_numbers(both):
    import numpy as np

    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(2, 64, device="cuda")
    want = ck.dropout(x, 0.5, 5, 6)
    a, b = both(lambda: ck.dropout(x, np.float32(0.5), np.int64(5), np.int32(6)))
    assert torch.equal(a, want) and torch.equal(b, want)
    h = torch.ones(2, 2, 64, device="cuda")
    a, b = both(lambda: ck.dropout(h, 0.5, np.uint64(5), np.int64(6), locked=np.bool_(True)))
    assert torch.equal(a, b) and torch.equal(a[0], a[1])
    a, b = both(lambda: ck.pick_tokens(x, temperature=np.float32(0.5), seed=np.int64(5), step=np.int64(6)))
    assert torch.equal(a, ck.pick_tokens(x, temperature=0.5, seed=5, step=6)) and torch.equal(a, b)


def test_numbers_that_32_bits_do_not_hold_are_refused(both):
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(2, 64, device="cuda")
    for kw in (dict(temperature=1e39), dict(temperature=1e-50), dict(repetition=1e39), dict(frequency=1e200),
               dict(presence=4e38)):
        for call in (ck.control_logits, ck.pick_tokens):
            def refused():
                with pytest.raises(ValueError):
                    call(x, **kw)
            both(refused)
    for kw in (dict(temperature=0), dict(temperature=3e38), dict(temperature=2e-45), dict(frequency=1e-60)):
        both(lambda: ck.control_logits(x, **kw))


def test_two_threads_on_two_streams():
    """Calls of several threads at once, each on a stream of its own, give what one gives."""
    import threading

    import sparse_graph_recurrent_gb300 as ck
    q, s, z = ck.int4_quantize(torch.randn(3000, 2000, device="cuda"), 64, symmetric=False)
    xs = [torch.randn(M, 2000, device="cuda") for M in (1, 20, 4, 33)]

    def work(x):
        h = ck.dropout(x, 0.3, 5, 6)
        y = ck.int4_matvec(h, q, s, z, group_size=64)
        return h, y, *ck.pick_tokens(y, temperature=0.7, seed=3, step=4, return_logits=True)

    want, wrong = [work(x) for x in xs], []
    torch.cuda.synchronize()

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                got = work(xs[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_out_made_in_inference_mode(both):
    """Written outside of it as well as inside: such tensors have no version to raise."""
    import sparse_graph_recurrent_gb300 as ck
    q, s, _ = ck.int4_quantize(torch.randn(64, 64, device="cuda"), 32)
    with torch.inference_mode():
        out, x = torch.empty(2, 64, device="cuda"), torch.randn(2, 64, device="cuda")
        inside = both(lambda: (ck.int4_matvec(x, q, s, group_size=32, out=out).clone(), ck.control_logits(x, out=out).clone()))
    outside = both(lambda: (ck.int4_matvec(x, q, s, group_size=32, out=out).clone(), ck.control_logits(x, out=out).clone()))
    assert all(torch.equal(u, v) for a, b in zip(inside, outside) for u, v in zip(a, b))
