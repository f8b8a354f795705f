"""Logit controls and the token they give, against numpy in 64 bits.

Tolerance of a controlled logit: at most six roundings of relative error
u = 2^-24 on terms no larger than m = |z| r + n |frequency| + |presence| + |bias|,
divided by the temperature: 6 u m / t, then one rounding to the logits' type.
A token has to be the largest score's up to that (two scores' worth, and the
noise's own 32-bit rounding, 4 u |noise| + 2^-22)."""
import numpy as np
import pytest
import torch

import readout_oracle as ro

pytestmark = pytest.mark.gpu

ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
INF = float("inf")


def pack(allowed):
    """int32 mask words of a bool array [..., V]."""
    V = allowed.shape[-1]
    pad = np.zeros((*allowed.shape[:-1], -(-V // 32) * 32), np.uint8)
    pad[..., :V] = allowed
    return np.ascontiguousarray(np.packbits(pad, axis=-1, bitorder="little")).view(np.int32)


def make(B, V, L, dtype=torch.float32, seed=0, allowed=0.5, bias="rows", ints=np.int64, rows=True):
    rng = np.random.default_rng(seed)
    n = rng.integers(0, L + 1, B).astype(ints)
    c = dict(
        history=(V * rng.random((B, L)) ** 3).astype(ints),
        history_len=n, prompt_len=(n * rng.random(B)).astype(ints),
        repetition=(1 + rng.random(B)).astype(np.float32),
        frequency=(0.5 * rng.random(B)).astype(np.float32),
        presence=rng.random(B).astype(np.float32),
        temperature=(0.5 + rng.random(B)).astype(np.float32))
    if not rows:
        for k in ("repetition", "frequency", "presence", "temperature"):
            c[k] = float(c[k][0])
    if bias != "none":
        c["bias"] = rng.normal(size=(B, V) if bias == "rows" else (V,)).astype(np.float32)
    if allowed:
        c["mask"] = pack(rng.random((B, V)) < allowed)
    logits = torch.from_numpy((3 * rng.normal(size=(B, V))).astype(np.float32)).to(dtype)
    return logits, c


def dev(c):
    return {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in c.items()}


def bounds(logits, c):
    z = np.abs(logits.double().numpy())
    B = z.shape[0]
    col = lambda k, d: np.broadcast_to(np.asarray(c.get(k, d), np.float64), (B,)).reshape(B, 1)  # noqa: E731
    r = np.maximum(col("repetition", 1.0), 1 / col("repetition", 1.0))
    L = c["history"].shape[1] if "history" in c else 0
    m = z * r + L * np.abs(col("frequency", 0.0)) + np.abs(col("presence", 0.0))
    m = m + (np.abs(c["bias"]) if "bias" in c else 0.0)
    t = col("temperature", 1.0)
    return 6 * 2.0 ** -24 * m / np.where(t > 0, t, 1.0) + 1e-30


def check_logits(out, logits, c):
    ref = ro.controlled(logits.double().numpy(), **c)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isneginf(ref), np.isneginf(got))
    fin = np.isfinite(ref)
    tol = bounds(logits, c) + ULP[logits.dtype] * np.abs(np.where(fin, ref, 0.0))
    if logits.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert (np.abs(got - ref)[fin] <= tol[fin]).all(), (np.abs(got - ref)[fin] / tol[fin]).max()
    return ref


def check_tokens(tokens, ref, logits, c, seed=None, step=0):
    B, V = ref.shape
    noise = np.zeros((B, V))
    if seed is not None:
        hot = np.broadcast_to(np.asarray(c.get("temperature", 1.0)), (B,)) > 0
        noise = ro.gumbel(B, V, seed, step) * hot[:, None]
    score = ref + noise
    slack = bounds(logits, c).max(1) + 4 * 2.0 ** -24 * np.abs(noise).max(1) + 2.0 ** -22
    got = tokens.cpu().numpy()
    assert got.dtype == np.int64 and got.shape == (B,)
    for b, want in enumerate(ro.pick(score)):
        if want < 0 or seed is None and got[b] == want:
            assert got[b] == want
        else:
            assert 0 <= got[b] < V and score[b, got[b]] >= score[b, want] - 2 * slack[b], b


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("B,V,L", [(1, 1, 1), (1, 256, 64), (3, 31, 0), (2, 33, 5), (4, 129, 300), (5, 1001, 40),
                                   (2, 5003, 700), (3, 20000, 100)])
def test_matches_the_definition(B, V, L, dtype):
    import sparse_graph_recurrent_gb300 as ck
    logits, c = make(B, V, L, dtype, seed=V + L)
    d = dev(c)
    x = logits.cuda()
    out = ck.control_logits(x, **d)
    ref = check_logits(out, logits, c)
    assert torch.equal(x.cpu(), logits)
    for seed in (None, 77):
        tokens = ck.pick_tokens(x, **d, seed=seed, step=3)
        check_tokens(tokens, ref, logits, c, seed, 3)
        again, z = ck.pick_tokens(x, **d, seed=seed, step=3, return_logits=True)
        assert torch.equal(tokens, again) and torch.equal(z, out)


@pytest.mark.parametrize("V", [70001, 262144])
def test_large_vocabularies(V):
    import sparse_graph_recurrent_gb300 as ck
    logits, c = make(2, V, 500, seed=V, bias="row", allowed=0)
    # the mask as words, shared by both rows; the oracle loops, so few tokens are forbidden there
    c["mask"] = np.full((-(-V // 32),), -1, np.int32)
    d = dev(c)
    out = ck.control_logits(logits.cuda(), **d)
    del c["mask"]
    ref = check_logits(out, logits, c)
    check_tokens(ck.pick_tokens(logits.cuda(), **d, seed=5, step=1), ref, logits, c, 5, 1)
    check_tokens(ck.pick_tokens(logits.cuda(), **d), ref, logits, c)


@pytest.mark.parametrize("leave", [[], ["history", "history_len", "prompt_len"], ["history_len"], ["prompt_len"],
                                   ["bias"], ["mask"], ["temperature"], ["repetition"], ["frequency", "presence"],
                                   ["history", "history_len", "prompt_len", "bias", "mask", "temperature",
                                    "repetition", "frequency", "presence"]])
def test_each_control_left_out(leave):
    import sparse_graph_recurrent_gb300 as ck
    for rows in (True, False):
        logits, c = make(3, 777, 90, seed=len(leave), rows=rows, ints=np.int32, bias="row")
        c = {k: v for k, v in c.items() if k not in leave}
        out = ck.control_logits(logits.cuda(), **dev(c))
        check_logits(out, logits, c)


def test_shared_and_strided_operands():
    import sparse_graph_recurrent_gb300 as ck
    logits, c = make(4, 333, 50, seed=11, bias="row")
    c["mask"] = c["mask"][0].copy()
    wide = torch.zeros(4, 350)
    wide[:, 7:340] = logits
    d = dev(c)
    h = torch.zeros(4, 61, dtype=torch.int64, device="cuda")
    h[:, 3:53] = d["history"]
    d["history"] = h[:, 3:53]
    out = torch.full((4, 341), 9.0, device="cuda")
    got, z = ck.pick_tokens(wide.cuda()[:, 7:340], **d, out=out[:, 5:338])
    ref = check_logits(z, logits, c)
    check_tokens(got, ref, logits, c)
    assert (out[:, :5] == 9).all() and (out[:, 338:] == 9).all()
    # in place
    x = logits.cuda()
    assert torch.equal(ck.control_logits(x, **d, out=x), z) and torch.equal(x, z)
    # rows of bias and mask with a pitch, and one row repeated by expand
    d["bias"] = torch.nn.functional.pad(d["bias"].expand(4, 333), (1, 2))[:, 1:334]
    d["mask"] = d["mask"].expand(4, -1)
    assert torch.equal(ck.control_logits(logits.cuda(), **d), z)


def test_padding_ids_and_lengths_are_clamped():
    import sparse_graph_recurrent_gb300 as ck
    logits, c = make(4, 100, 40, seed=12)
    c["history"][:, 5:9] = [-1, 100, 2 ** 40, -2 ** 40]
    c["history_len"] = np.array([-3, 0, 40, 10 ** 9])
    c["prompt_len"] = np.array([0, 5, 10 ** 9, -7])
    check_logits(ck.control_logits(logits.cuda(), **dev(c)), logits, c)


def test_long_history_of_few_tokens():
    """Counts far above what 16 bits hold, all on a few tokens."""
    import sparse_graph_recurrent_gb300 as ck
    B, V, L = 2, 500, 200_001
    logits = torch.randn(B, V)
    history = torch.zeros(B, L, dtype=torch.int32)
    history[:, ::2] = 499
    c = dict(history=history.numpy(), frequency=0.25, presence=1.0, repetition=1.5,
             prompt_len=np.array([1, 100_000], np.int32))
    check_logits(ck.control_logits(logits.cuda(), **dev(c)), logits, c)


def test_rows_with_nothing_left_and_special_values():
    import sparse_graph_recurrent_gb300 as ck
    V = 300
    logits = torch.randn(8, V)
    allowed = np.ones((8, V), bool)
    allowed[0] = False                            # nothing allowed
    allowed[1] = False
    allowed[1, 299] = True                        # one token
    logits[2] = -INF                              # nothing above -inf
    logits[3, 17] = logits[3, 200] = INF          # the lower of two infinities
    logits[4] = float("nan")                      # nothing but NaN
    logits[5, ::2] = float("nan")                 # NaN is never picked
    allowed[6, 5:] = False
    logits[6, 5:] = float("nan")                  # NaN in masked places does no harm
    logits[7] = torch.finfo(torch.float32).min    # the type's lowest value is a value
    x, m = logits.cuda(), torch.from_numpy(pack(allowed)).cuda()
    for seed in (None, 3):
        tokens, z = ck.pick_tokens(x, mask=m, seed=seed, return_logits=True)
        t = tokens.cpu().tolist()
        assert t[0] == -1 and t[1] == 299 and t[2] == -1 and t[3] == 17 and t[4] == -1
        assert t[5] % 2 == 1 and 0 <= t[6] < 5
        assert t[7] == 0 if seed is None else 0 <= t[7] < V
        want = torch.where(torch.from_numpy(allowed), logits, -INF)
        assert torch.equal(torch.nan_to_num(z.cpu(), 5.0), torch.nan_to_num(want, 5.0))


def test_ties_go_to_the_lowest_token():
    import sparse_graph_recurrent_gb300 as ck
    for V in (7, 1000, 40000):
        x = torch.zeros(3, V, device="cuda")
        x[1] = -0.0
        x[1, V // 2:] = 0.0   # -0 and 0 are equal
        x[2, V // 3:] = 1.5
        assert ck.pick_tokens(x).tolist() == [0, 0, V // 3]


def test_temperature_zero_is_greedy():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(4, 5000, device="cuda")
    t = torch.tensor([0.0, 1.0, 0.0, 2.0], device="cuda")
    tok, z = ck.pick_tokens(x, temperature=t, seed=9, step=1, return_logits=True)
    best = x.argmax(1)
    assert tok[0] == best[0] and tok[2] == best[2]
    assert torch.equal(z[0], x[0]) and torch.equal(z[3], x[3] / 2)
    assert torch.equal(ck.pick_tokens(x, temperature=0.0, seed=9), best)


def test_draws_follow_the_softmax():
    """40,000 draws from six tokens: each count within 6 standard deviations."""
    import sparse_graph_recurrent_gb300 as ck
    n = 40000
    z = torch.tensor([0.0, 1.0, -1.0, 2.0, -INF, 0.5], device="cuda")
    p = torch.softmax(z.double() / 0.7, 0).cpu().numpy()
    got = torch.cat([ck.pick_tokens(z.expand(10000, 6), temperature=0.7, seed=4, step=s) for s in range(4)])
    count = np.bincount(got.cpu().numpy(), minlength=6)
    assert count[4] == 0
    assert (np.abs(count - n * p) <= 6 * np.sqrt(n * p * (1 - p)) + 1e-9).all()


def test_element_indexes_past_32_bits():
    """40,000 rows of 131,072 tokens, one row of logits shared by all: the noise of the
    last rows is that of elements past 2^32."""
    import sparse_graph_recurrent_gb300 as ck
    B, V = 40_000, 131_072
    z = torch.randn(V, device="cuda")
    got = ck.pick_tokens(z.expand(B, V), seed=3, step=2)
    for b in (0, 16384, 32768, B - 1):
        w = ro.philox_words(np.arange(b * V, (b + 1) * V), 3, 2).astype(np.float64)
        u = np.minimum(w * 2.0 ** -32 + 2.0 ** -33, 1 - 2.0 ** -24)
        score = z.double().cpu().numpy() - np.log(-np.log1p(-u))
        assert score[int(got[b])] >= score.max() - 1e-5


def test_in_place_and_many_rows():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.randn(70, 9000, device="cuda") * 2
    t = torch.rand(70, device="cuda") + 0.5
    want, z = ck.pick_tokens(x, temperature=t, seed=8, step=4, return_logits=True)
    y = x.clone()
    got, same = ck.pick_tokens(y, temperature=t, seed=8, step=4, out=y)
    assert torch.equal(got, want) and torch.equal(y, z) and same is y
    assert torch.equal(ck.pick_tokens(x, temperature=t, seed=8, step=4), want)


def test_step_on_the_device_capture_and_streams():
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck
    x = torch.randn(5, 3001, device="cuda")
    step = torch.tensor([4], dtype=torch.int64, device="cuda")
    want = [ck.pick_tokens(x, seed=1, step=k) for k in range(4, 9)]
    assert torch.equal(ck.pick_tokens(x, seed=1, step=step), want[0])
    assert not all(torch.equal(w, want[0]) for w in want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ck.pick_tokens(x, seed=1, step=5)
    s.synchronize()
    assert torch.equal(got, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok = ck.pick_tokens(x, seed=1, step=step)
        _ck.ck_step_advance(step)
    for k in range(4):
        g.replay()
        assert torch.equal(tok, want[k])


def test_refusals():
    import sparse_graph_recurrent_gb300 as ck
    logits, c = make(2, 64, 10)
    d, x = dev(c), logits.cuda()
    ck.pick_tokens(x, **d)
    for bad in (dict(history=d["history"].float()), dict(history=d["history"][:1]),
                dict(history_len=d["history_len"].int()), dict(prompt_len=d["prompt_len"][:1]),
                dict(history=None), dict(repetition=0.0), dict(repetition=-1.0), dict(temperature=-0.5),
                dict(temperature=float("nan")), dict(frequency=INF), dict(presence=d["presence"].double()),
                dict(presence=d["presence"][:1]), dict(bias=d["bias"][:, :63]), dict(bias=d["bias"].half()),
                dict(mask=d["mask"].long()), dict(mask=d["mask"][:, :1]), dict(out=torch.empty(2, 64)),
                dict(out=x.half())):
        with pytest.raises(ValueError):
            ck.pick_tokens(x, **{**d, **bad})
    for v in (x[0], x.double(), x.clone().requires_grad_()):
        with pytest.raises(ValueError):
            ck.control_logits(v)
    with pytest.raises(ck.CKError):
        ck.control_logits(x[:, :0])
    with pytest.raises(ValueError):
        ck.pick_tokens(x, seed=1, step=torch.tensor([1]))
    assert ck.pick_tokens(x[:0]).shape == (0,)


def test_temperatures_at_the_ends_of_their_type():
    """Where 1 / T is no normal number: z / T within an ulp of it, tokens as z / T + noise orders them."""
    import sparse_graph_recurrent_gb300 as ck
    temps = np.array([1e-39, 1e-44, 2.5e38, 3.4e38, np.inf, 1e37, 1e-37], np.float32)
    B, V = len(temps), 300
    rng = np.random.default_rng(8)
    z = rng.standard_normal((B, V)).astype(np.float32)
    z[:, ::7] = 0.0
    z[0, :] = np.minimum(z[0], 0.0)  # the best is 0 / T
    z[2] *= np.float32(1e38)
    with np.errstate(over="ignore", invalid="ignore"):
        want = z / temps[:, None]
    x, t = torch.from_numpy(z).cuda(), torch.from_numpy(temps).cuda()
    got = ck.control_logits(x, temperature=t).cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert (np.abs(got - want)[fin] <= 2.0 ** -22 * np.abs(want)[fin] + 2.0 ** -148).all()
    assert ck.pick_tokens(x, temperature=t).cpu().tolist() == want.argmax(1).tolist()
    score = want.astype(np.float64) + ro.gumbel(B, V, 9, 2)
    tokens = ck.pick_tokens(x, temperature=t, seed=9, step=2).cpu().numpy()
    for b in range(B):
        best = score[b].max()
        assert score[b, tokens[b]] == best or best - score[b, tokens[b]] < 1e-5, b


@pytest.mark.parametrize("L", [32767, 32768, 40000])
@pytest.mark.parametrize("ints", [np.int32, np.int64])
def test_one_token_all_along_a_long_history(L, ints):
    """Counts up to the history's length, on both sides of where they are kept in more bits."""
    import sparse_graph_recurrent_gb300 as ck
    V, token = 9001, 8070
    x = torch.zeros(2, V)
    x[:, token] = 3.0
    history = torch.full((2, L), token, dtype=torch.from_numpy(np.zeros(1, ints)).dtype)
    prompt = torch.tensor([0, L - 1], dtype=history.dtype)
    out = ck.control_logits(x.cuda(), history=history.cuda(), prompt_len=prompt.cuda(), repetition=2.0,
                            frequency=0.5, presence=0.25).cpu()
    assert out[0, token] == 1.5 - (L * 0.5 + 0.25) and out[1, token] == 1.5 - 0.75
    out[:, token] = 0.0
    assert not out.any()


@pytest.mark.parametrize("V", [8064, 8065, 16256, 16257, 33000])
@pytest.mark.parametrize("dtype", list(ULP))
def test_many_rows_and_equal_scores(V, dtype):
    """Whole waves of rows; half of a row shares its highest logit: the lowest index, at any temperature."""
    import sparse_graph_recurrent_gb300 as ck
    B = 700
    x = torch.zeros(B, V, dtype=dtype)
    first = torch.arange(B) * 11 % (V // 2)
    top = torch.arange(V)[None, :] >= first[:, None]
    x[top] = 5.0
    for temperature in (1.0, 0.7, 0.0):
        tokens = ck.pick_tokens(x.cuda(), temperature=temperature)
        assert torch.equal(tokens.cpu(), first)


def test_ties_of_scores_that_overflow():
    """Logits whose quotients by the temperature are infinite are equal: the lowest token, at
    temperatures whose reciprocal is a normal number too, in one slice or several."""
    import sparse_graph_recurrent_gb300 as ck
    x = torch.tensor([[70.0, 100.0]], device="cuda")
    for seed in (None, 5):
        assert ck.pick_tokens(x, temperature=2e-37, seed=seed).tolist() == [0]
    for V in (300, 20000, 140000):
        x = torch.randn(6, V, device="cuda")
        x[:, V // 2] = 80.0                                     # the first that overflows
        x[:, V // 2 + 5 :: 7] = 90.0
        x[:, V - 1] = 3e38
        x[5] = torch.linspace(69.0, 400.0, V, device="cuda")    # near the end of the type, then past it
        for t in (1.5e-37, 2e-37, 2.0349e-37):
            with np.errstate(over="ignore"):
                z = x.cpu().numpy() / np.float32(t)
            want = z.argmax(1).tolist()
            assert want[:5] == [V // 2] * 5 and np.isinf(z[5].max())
            for seed in (None, 5):
                for kw in (dict(temperature=t), dict(temperature=torch.full((6,), t, device="cuda"))):
                    assert ck.pick_tokens(x, **kw, seed=seed, step=2).tolist() == want
                    tok, out = ck.pick_tokens(x, **kw, seed=seed, step=2, return_logits=True)
                    assert tok.tolist() == want and torch.isinf(out.max(1).values).all()
    x = torch.zeros(2, 9000, device="cuda")
    x[0, 4000:], x[1, 7::9] = 3e38, 2e38                        # at an ordinary temperature
    assert ck.pick_tokens(x, temperature=0.5).tolist() == [4000, 7]
    assert ck.pick_tokens(x, temperature=0.5, seed=1).tolist() == [4000, 7]


@pytest.mark.parametrize("V", [300, 20001])
def test_fp32_logits_are_the_quotient(V):
    """Of 32-bit logits and no other control the result is z / T, rounded once."""
    import sparse_graph_recurrent_gb300 as ck
    rng = np.random.default_rng(V)
    z = (3 * rng.standard_normal((40, V))).astype(np.float32)
    t = (0.1 + 2 * rng.random(40)).astype(np.float32)
    x, temps = torch.from_numpy(z).cuda(), torch.from_numpy(t).cuda()
    want = z / t[:, None]
    assert np.array_equal(ck.control_logits(x, temperature=temps).cpu().numpy(), want)
    for seed in (None, 4):
        tokens, out = ck.pick_tokens(x, temperature=temps, seed=seed, return_logits=True)
        assert np.array_equal(out.cpu().numpy(), want)
        if seed is None:
            assert tokens.cpu().tolist() == want.argmax(1).tolist()
    assert np.array_equal(ck.control_logits(x, temperature=0.7).cpu().numpy(), z / np.float32(0.7))
    assert torch.equal(ck.control_logits(x, temperature=1.0), x)


def test_fp32_quotients_over_the_whole_type():
    """Any 32 bits by any temperature: the division's result, bit for bit but for NaN's payload."""
    import sparse_graph_recurrent_gb300 as ck
    g = torch.Generator().manual_seed(3)
    bits = lambda *n: torch.randint(-2 ** 31, 2 ** 31, n, generator=g).int().view(torch.float32)  # noqa: E731
    B, V = 400, 40000
    t = bits(B).abs()
    t[torch.isnan(t)] = 0.7
    t[::2] = torch.rand(B, generator=g)[::2] * 3 + 0.01            # half of them ordinary
    t[:8] = torch.tensor([1 - 2.0 ** -24, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 0.75, 1.5, 2.0, 2.0 ** -126, 2.0 ** 127])
    x = bits(B, V)
    near = torch.randn(B // 2, V, generator=g) * 5
    x[::2] = near
    x[:, :6] = torch.tensor([0.0, -0.0, INF, -INF, 1e-45, 3.4e38])
    want = torch.where(t[:, None] > 0, x.cuda().cpu().div(t[:, None]), x)
    want_dev = torch.where(t.cuda()[:, None] > 0, x.cuda() / t.cuda()[:, None], x.cuda())
    out = ck.control_logits(x.cuda(), temperature=t.cuda())
    for w in (want.cuda(), want_dev):
        nan = torch.isnan(w)
        assert torch.equal(torch.isnan(out), nan)
        assert torch.equal(out[~nan].view(torch.int32), w[~nan].view(torch.int32))
