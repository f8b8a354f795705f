"""The 4-bit product and its quantiser against numpy in 64 bits.

Tolerance of the product, from its formula: K products added in 32-bit floats in
any order are off by at most K u sum |w| |x| with u = 2^-24; tensor-core sums may
truncate, twice that; scales and the split of x add a few u more; the result is
rounded once to x's type (half a unit in the last place)."""
import numpy as np
import pytest
import torch

import readout_oracle as ro

pytestmark = pytest.mark.gpu

ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def case(M, K, V, group, dtype, scale_dtype=None, zeros=True, seed=0, pad_rows=0):
    rng = np.random.default_rng(seed)
    n, G = (K + 1) // 2, -(-K // group)
    buf = torch.from_numpy(rng.integers(0, 256, (V, -(-n // 16) * 16 + 16 * pad_rows), dtype=np.uint8)).cuda()
    return dict(
        x=torch.from_numpy(np.tanh(rng.normal(size=(M, K))).astype(np.float32)).to(dtype).cuda(),
        qweight=buf[:, :n],
        scales=torch.from_numpy((0.01 + rng.random((V, G)) / np.sqrt(K)).astype(np.float32)).to(scale_dtype or dtype).cuda(),
        zeros=torch.from_numpy(rng.integers(0, 16, (V, G), dtype=np.uint8)).cuda() if zeros else None)


def check(y, c, group, bias=None):
    x = c["x"].double().cpu().numpy().reshape(-1, c["x"].shape[-1])
    K = x.shape[1]
    w = ro.dequantize(c["qweight"].cpu().numpy(), c["scales"].double().cpu().numpy(),
                      None if c["zeros"] is None else c["zeros"].cpu().numpy(), K, group)
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        ref, mag = ref + bias.double().cpu().numpy(), mag + np.abs(bias.double().cpu().numpy())
    tol = (2 * K + 16) * 2.0 ** -24 * mag + ULP[c["x"].dtype] * np.abs(ref) + 1e-30
    if c["x"].dtype == torch.float16:
        tol += 2.0 ** -25  # subnormal results
    got = y.double().cpu().numpy().reshape(ref.shape)
    worst = (np.abs(got - ref) / tol).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,V", [(1, 1, 1), (1, 2, 17), (1, 31, 5), (1, 33, 16), (2, 255, 33), (3, 257, 100),
                                   (1, 5000, 256), (8, 1024, 64), (5, 8193, 15), (1, 20001, 7)])
def test_matches_the_definition(M, K, V, group, dtype):
    import sparse_graph_recurrent_gb300 as ck
    c = case(M, K, V, group, dtype, seed=M + K + V + group)
    check(ck.int4_matvec(**c, group_size=group), c, group)


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 10, 12, 16, 17, 20, 24, 31, 32, 33, 48, 64, 65, 100, 130])
def test_rows_of_x(M, dtype):
    import sparse_graph_recurrent_gb300 as ck
    c = case(M, 700, 150, 64, dtype, zeros=M % 2 == 0, seed=M)
    check(ck.int4_matvec(**c, group_size=64), c, 64)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,M", [(torch.float32, 5), (torch.float32, 11), (torch.float32, 21), (torch.float32, 32),
                                     (torch.bfloat16, 17), (torch.bfloat16, 33), (torch.bfloat16, 96),
                                     (torch.float16, 32), (torch.float16, 64), (torch.float16, 70)])
def test_batches_at_every_width(dtype, M, group, zeros):
    """Every width and group of the product for batches; a block of rows that is not
    full, a half of it that is empty, K that ends inside every tile."""
    import sparse_graph_recurrent_gb300 as ck
    for K, V in ((1, 3), (65, 127), (700, 300), (1217, 129)):
        c = case(M, K, V, group, dtype, zeros=zeros, seed=M + K, pad_rows=V % 2)
        check(ck.int4_matvec(**c, group_size=group), c, group)


@pytest.mark.parametrize("dtype,M", [(torch.float32, 20), (torch.float16, 40)])
@pytest.mark.parametrize("K,V", [(40000, 100), (9000, 2000), (300, 45000)])
def test_batches_in_one_run_of_k_and_in_many(K, V, dtype, M):
    import sparse_graph_recurrent_gb300 as ck
    c = case(M, K, V, 128, dtype, seed=K)
    bias = torch.randn(V, device="cuda")
    a = ck.int4_matvec(**c, bias=bias)
    check(a, c, 128, bias)
    assert torch.equal(ck.int4_matvec(**c, bias=bias), a)


def test_batch_side_stream_and_capture():
    import sparse_graph_recurrent_gb300 as ck
    c = case(20, 3000, 500, 64, torch.float32, seed=4)
    a = ck.int4_matvec(**c, group_size=64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = ck.int4_matvec(**c, group_size=64)
    s.synchronize()
    assert torch.equal(a, b)
    out = torch.empty_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.int4_matvec(**c, group_size=64, out=out)
    c["x"].mul_(0.5)
    g.replay()
    assert torch.equal(out, a * 0.5)


def test_a_wait_that_runs_out_leaves_nan_and_a_usable_device():
    """The batch product's waits are bounded: with an arrival asked for that never comes
    all of them give up, y is NaN, and the next call is right."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    c = case(8, 2000, 600, 128, torch.float32, seed=6)
    _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 1)
    _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 2_000_000)
    try:
        y = ck.int4_matvec(**c)
        torch.cuda.synchronize()
        assert torch.isnan(y).all()
    finally:
        _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 0)
        _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 4_000_000_000)
    check(ck.int4_matvec(**c), c, 128)


@pytest.mark.parametrize("M", [2, 8])
def test_weights_past_two_gigabytes(M):
    """Rows whose bytes lie past 2^31; the last ones are compared."""
    import sparse_graph_recurrent_gb300 as ck
    K, V, n = 65536, 70000, 64
    small = case(M, K, n, 128, torch.bfloat16, seed=7)
    q = torch.zeros(V, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(V, K // 128, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(V, K // 128, dtype=torch.uint8, device="cuda")
    q[-n:], s[-n:], z[-n:] = small["qweight"], small["scales"], small["zeros"]
    y = ck.int4_matvec(small["x"], q, s, z)
    check(y[:, -n:].contiguous(), small, 128)
    assert not y[:, :-n].any()


@pytest.mark.parametrize("M,V", [(1, 40000), (4, 9001), (32, 5000), (20, 2500)])
def test_many_outputs(M, V):
    import sparse_graph_recurrent_gb300 as ck
    c = case(M, 300, V, 128, torch.float32, seed=V)
    check(ck.int4_matvec(**c, group_size=128), c, 128)


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("M", [1, 4, 20])
def test_long_axis(M, dtype):
    import sparse_graph_recurrent_gb300 as ck
    c = case(M, 211577, 40, 128, dtype, seed=M)
    check(ck.int4_matvec(**c, group_size=128), c, 128)


@pytest.mark.parametrize("sdt", list(ULP))
@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("group", [32, 128])
def test_types_strides_bias_and_shapes(group, dtype, sdt):
    import sparse_graph_recurrent_gb300 as ck
    c = case(6, 517, 90, group, dtype, scale_dtype=sdt, seed=9, pad_rows=3)
    wide = torch.zeros(90, c["scales"].shape[1] + 3, dtype=sdt, device="cuda")
    wide[:, :-3] = c["scales"]
    c["scales"] = wide[:, :-3]
    zw = torch.zeros(90, c["zeros"].shape[1] + 5, dtype=torch.uint8, device="cuda")
    zw[:, 5:] = c["zeros"]
    c["zeros"] = zw[:, 5:]
    xw = torch.full((6, 530), float("nan"), dtype=dtype, device="cuda")
    xw[:, 1:518] = c["x"]
    c["x"] = xw[:, 1:518]
    bias = torch.randn(90, device="cuda")
    check(ck.int4_matvec(**c, bias=bias, group_size=group), c, group, bias)
    out = torch.full((6, 100), 7.0, dtype=dtype, device="cuda")
    assert ck.int4_matvec(**c, bias=bias, group_size=group, out=out[:, 4:94]).data_ptr() == out[:, 4:].data_ptr()
    check(out[:, 4:94].contiguous(), c, group, bias)
    assert (out[:, :4] == 7).all() and (out[:, 94:] == 7).all()
    x = c.pop("x")
    y3 = ck.int4_matvec(x.reshape(2, 3, 517), **c, group_size=group)
    assert y3.shape == (2, 3, 90)
    y1 = ck.int4_matvec(x[5], **c, group_size=group)
    assert y1.shape == (90,)
    xt = x.t().contiguous().t()  # K not dense
    assert torch.equal(ck.int4_matvec(xt, **c, group_size=group), y3.view(6, 90))
    assert ck.int4_matvec(x[:0], **c, group_size=group).shape == (0, 90)


def test_tail_bytes_are_not_used():
    """The spare nibble of an odd K, what follows a row and what follows x's row change nothing."""
    import sparse_graph_recurrent_gb300 as ck
    c = case(3, 333, 50, 64, torch.float32, seed=1)
    a = ck.int4_matvec(**c, group_size=64)
    base = c["qweight"]._base if c["qweight"]._base is not None else c["qweight"]
    c["qweight"][:, -1] ^= 0xF0
    full = torch.as_strided(base, (50, base.stride(0)), (base.stride(0), 1))
    full[:, c["qweight"].shape[1]:] ^= 0xFF
    assert torch.equal(ck.int4_matvec(**c, group_size=64), a)


def test_large_and_small_values():
    """x over the range of float32 and of bfloat16, rows kept apart."""
    import sparse_graph_recurrent_gb300 as ck
    for dtype in (torch.float32, torch.bfloat16):
        for M in (4, 20):
            c = case(M, 640, 48, 32, dtype, scale_dtype=torch.float32, seed=2)
            mag = torch.tensor([1e-30, 1e-12, 1.0, 1e30], device="cuda").repeat(M // 4).view(-1, 1)
            c["x"] = (c["x"].float() * mag).to(dtype)
            check(ck.int4_matvec(**c, group_size=32), c, 32)
            # one large element in a row of small ones
            c["x"][:, 100] = 1e4
            check(ck.int4_matvec(**c, group_size=32), c, 32)


def test_not_finite_x_stays_in_its_row():
    import sparse_graph_recurrent_gb300 as ck
    for dtype in ULP:
        c = case(5, 400, 33, 64, dtype, seed=3)
        clean = ck.int4_matvec(**c, group_size=64)
        c["x"][1, 7], c["x"][3, 399] = float("inf"), float("nan")
        y = ck.int4_matvec(**c, group_size=64)
        assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
        assert not torch.isfinite(y[1]).any() or not torch.isfinite(y[1]).all()
        assert torch.isnan(y[3]).all()


def test_side_stream_capture_and_repeat():
    import sparse_graph_recurrent_gb300 as ck
    c = case(4, 3000, 500, 128, torch.float32, seed=4)
    a = ck.int4_matvec(**c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = ck.int4_matvec(**c)
    s.synchronize()
    assert torch.equal(a, b)  # the same sums in the same order
    out = torch.empty_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.int4_matvec(**c, out=out)
    c["x"].mul_(0.5)
    g.replay()
    assert torch.equal(out, a * 0.5)


def reference_quantize(w, group, symmetric, scale_dtype):
    V, K = w.shape
    G = -(-K // group)
    pad = np.zeros((V, G * group))
    pad[:, :K] = w
    pad = pad.reshape(V, G, group)
    lo, hi = np.minimum(pad.min(-1), 0), np.maximum(pad.max(-1), 0)
    s = np.maximum(-lo / 8, hi / 7) if symmetric else (hi - lo) / 15
    return s


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", list(ULP))
def test_quantize(dtype, group, symmetric):
    """Scales as the formula has them, and every weight within half a step of its
    nibble's value (plus what rounding the scale to its type moves the ends of the
    range: 15 steps times half a unit)."""
    import sparse_graph_recurrent_gb300 as ck
    for V, K in ((1, 1), (5, 33), (20, 515), (3, 1024)):
        w = torch.from_numpy(np.random.default_rng(K).normal(size=(V, K)).astype(np.float32)).to(dtype).cuda()
        w[0] = 0
        if V > 1:
            w[1] = w[1].abs() + 1
            w[2] = -w[2].abs() - 1
        q, s, z = ck.int4_quantize(w, group, symmetric)
        assert q.shape == (V, (K + 1) // 2) and (V == 1 or q.stride(0) % 16 == 0)
        assert (z is None) == symmetric and s.dtype == dtype
        want = reference_quantize(w.double().cpu().numpy(), group, symmetric, dtype)
        sd = s.double().cpu().numpy()
        # fp32 arithmetic of three roundings, then one rounding to the scale's type
        assert np.abs(sd - want).max() <= (ULP[dtype] + 3 * 2.0 ** -24) * np.abs(want).max() + 2.0 ** -25
        back = ro.dequantize(q.cpu().numpy(), sd, None if z is None else z.cpu().numpy(), K, group)
        step = np.repeat(sd, group, axis=1)[:, :K]
        # symmetric: an end of the range may round to one nibble past it and be clamped
        err = np.abs(back - w.double().cpu().numpy())
        slack = 0.5 + 15 * (ULP[dtype] + 3 * 2.0 ** -24) + (0.0 if symmetric else 0.5)
        assert (err <= slack * step + 1e-30).all()
        assert not back[0].any()


def test_quantize_then_multiply_and_not_finite_weights():
    import sparse_graph_recurrent_gb300 as ck
    w = torch.randn(64, 300, device="cuda") / 17
    x = torch.tanh(torch.randn(2, 300, device="cuda"))
    for symmetric in (True, False):
        q, s, z = ck.int4_quantize(w, 32, symmetric, scale_dtype=torch.float16)
        check(ck.int4_matvec(x, q, s, z, group_size=32), dict(x=x, qweight=q, scales=s, zeros=z), 32)
    w[3, 40] = float("inf")
    w[5, 299] = float("nan")
    _, s, _ = ck.int4_quantize(w.t().contiguous().t(), 32)
    bad = torch.isnan(s)
    assert bad[3, 1] and bad[5, 9] and int(bad.sum()) == 2
    assert ck.int4_quantize(w[:0], 32)[0].shape == (0, 150)


def test_refusals():
    import sparse_graph_recurrent_gb300 as ck
    c = case(2, 64, 8, 32, torch.float32)
    ok = dict(c, group_size=32)
    ck.int4_matvec(**ok)
    for bad in (dict(group_size=48), dict(x=c["x"].double()), dict(x=c["x"][:, :62]),
                dict(scales=c["scales"][:, :1]), dict(scales=c["scales"].double()),
                dict(zeros=c["zeros"].int()), dict(zeros=c["zeros"][:4]),
                dict(qweight=c["qweight"].int()), dict(bias=torch.zeros(7, device="cuda")),
                dict(bias=torch.zeros(8, device="cuda", dtype=torch.float16)),
                dict(out=torch.zeros(2, 9, device="cuda")), dict(x=c["x"].clone().requires_grad_()),
                dict(x=c["x"][:, :0])):
        with pytest.raises(ValueError):
            ck.int4_matvec(**{**ok, **bad})
    tight = torch.zeros(8 * 40 + 16, dtype=torch.uint8, device="cuda")
    for q in (torch.as_strided(tight, (8, 32), (40, 1)), torch.as_strided(tight, (8, 32), (32, 1), 8)):
        with pytest.raises(ck.CKError) as e:
            ck.int4_matvec(**{**ok, "qweight": q})
        assert e.value.name == "CK_ERR_INVALID_ARG"
    with pytest.raises(ValueError):
        ck.int4_quantize(torch.zeros(4, 64, device="cuda"), 48)
    with pytest.raises(ValueError):
        ck.int4_quantize(torch.zeros(4, device="cuda"))


@pytest.mark.parametrize("M", [4, 20])
def test_a_named_stream_while_the_current_one_is_busy(M):
    """Blocks that the current stream has given back, but still writes, are not the
    workspace of a product on another stream."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    c = case(M, 3000, 2000, 128, torch.float32, seed=4)
    want = ck.int4_matvec(**c)
    need = _ck.ck_int4_workspace_size(torch.float32, M, 3000, 2000, 128)
    assert need > 0
    s = torch.cuda.Stream()
    ys = [torch.empty_like(want) for _ in range(20)]
    torch.cuda.synchronize()
    for _ in range(400):
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0x7f)
    for y in ys:
        _ck.ck_int4_matvec(c["x"], c["qweight"], c["scales"], c["zeros"], None, 128, y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


# (M, K, V, dtype): 12 warps with whole tiles, 12 with the joining kernel, two column tiles,
# slabs of a long K, 16 warps with a long run
@pytest.mark.parametrize("M,K,V,dtype", [(1, 5000, 256, torch.float32), (4, 3000, 500, torch.float32),
                                         (16, 2000, 3000, torch.bfloat16), (4, 211577, 40, torch.float32),
                                         (1, 40000, 16384, torch.float16)])
def test_a_wait_that_runs_out_with_few_rows(M, K, V, dtype):
    """As for batches: every wait for weights gives up, y is NaN wherever sums meet, and the
    next call is right."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    c = case(M, K, V, 128, dtype, seed=6)
    _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 1)
    _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 2_000_000)
    try:
        ys = [ck.int4_matvec(**c) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.isnan(y).all() for y in ys)
    finally:
        _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 0)
        _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 4_000_000_000)
    check(ck.int4_matvec(**c), c, 128)


@pytest.mark.parametrize("K", [64, 600, 1217, 20000])
def test_a_wait_that_runs_out_with_copies_on_their_way(K):
    """Short runs of K, whose copies have all been asked for when the warps that would take
    them up give up: the block waits for them before it ends, and other calls follow at once."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    c, d = case(20, K, 300, 64, torch.float32, seed=6), case(3, 5000, 3000, 64, torch.float32, seed=7)
    want = ck.int4_matvec(**d, group_size=64)
    torch.cuda.synchronize()
    _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 100_000)
    try:
        for _ in range(5):
            _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 1)
            y = ck.int4_matvec(**c, group_size=64)
            _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 0)
            _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 4_000_000_000)
            assert torch.equal(ck.int4_matvec(**d, group_size=64), want)
            assert torch.isnan(y).all()
            _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 100_000)
    finally:
        _ck.ck_set_option(_ck.OPT_TEST_BARRIER_EXTRA, 0)
        _ck.ck_set_option(_ck.OPT_BARRIER_TIMEOUT_NS, 4_000_000_000)
    check(ck.int4_matvec(**c, group_size=64), c, 64)


@pytest.mark.parametrize("K", [5000, 64, 333, 1])
@pytest.mark.parametrize("symmetric", [True, False])
def test_weights_that_were_copied(K, symmetric):
    """clone, to and a state_dict's copy make the rows of the weights dense; the product is the same."""
    import sparse_graph_recurrent_gb300 as ck
    q, s, z = ck.int4_quantize(torch.randn(70, K, device="cuda"), 32, symmetric)
    for M in (1, 20):
        x = torch.randn(M, K, device="cuda")
        want = ck.int4_matvec(x, q, s, z, group_size=32)
        for c in (q.clone(), q.cpu().cuda(), q.contiguous(), torch.cat([q[:40], q[40:]])):
            assert torch.equal(ck.int4_matvec(x, c, s, z, group_size=32), want)
            again = ck.int4_rows(c)
            assert torch.equal(again, q) and again.stride(0) % 16 == 0 and again.data_ptr() % 16 == 0
            assert torch.equal(ck.int4_matvec(x, again, s, z, group_size=32), want)
    assert ck.int4_rows(q) is q
