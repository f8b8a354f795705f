"""The operators of a trained and answering recurrent model at the sizes they are used
at: a gated linear recurrence over long sequences with its gradients, the global norm
of many gradients and their clipping, and a beam search's selection with the reordering
of its beams' states.

Each case runs either in plain form (elementary torch operations in 32 bits, in 64 for a
beam's scores, `own = False`) or through this framework's entry points (`own = True`).
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
_DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # -- gated linear recurrence over [T, B, N] -----------------------------------------------
        # one input step of a few sequences being answered: latency of a call
        dict(name="gated_step_8", op="gated", T=1, B=8, N=256, dtype="float32", form="leak",
             lengths=False, grad=False),
        # the FlyGPT window as a training step sees it, forward and gradients
        dict(name="gated_flygpt", op="gated", T=64, B=32, N=5000, dtype="float32", form="leak",
             lengths=False, grad=True),
        # the ragged workload's batch of 20, an odd width, sequences of different lengths
        dict(name="gated_ragged_half", op="gated", T=96, B=20, N=4999, dtype="float16", form="leak",
             lengths=True, grad=True),
        # one long text through a narrow layer: few channels, the long axis split
        dict(name="gated_long_bf16", op="gated", T=65536, B=1, N=256, dtype="bfloat16", form="decay",
             lengths=False, grad=True),
        # -- global gradient norm and clipping ----------------------------------------------------
        # the tiny workload's edge values, leaks and biases: the smallest training step
        dict(name="clip_tiny", op="clip", sizes="tiny", count=3, ratio=0.5, mixed=False),
        # a model of many parameters, from single numbers up, in two types
        dict(name="clip_many", op="clip", sizes="many", count=400, ratio=0.5, mixed=True),
        # the whole connectome's edges, leaks and biases with a byte readout in 16 bits
        dict(name="clip_connectome", op="clip", sizes="connectome", count=4, ratio=2.0, mixed=True),
        # -- a beam search's step: selection, and the beams' states reordered ---------------------
        # one byte-level sequence with four beams: latency of an answering loop
        dict(name="beam_bytes_4", op="beam", B=1, K=4, V=256, dtype="float32", N=5000, L=64, ended=0.0),
        # eight sequences over a vocabulary of words, some beams at their end
        dict(name="beam_words_8", op="beam", B=8, K=8, V=32000, dtype="float32", N=5000, L=128, ended=0.2),
        # many beams, a large vocabulary, the wide workload's states
        dict(name="beam_large_16", op="beam", B=16, K=16, V=131072, dtype="bfloat16", N=20000, L=1024,
             ended=0.1),
        # -- reordering alone ---------------------------------------------------------------------
        # FlyGPT states of eight sequences with four beams and their texts
        dict(name="reorder_flygpt", op="reorder", B=8, K=4, N=5000, dtype="float32", L=256),
        # states of the whole connectome, rows of an odd length
        dict(name="reorder_connectome", op="reorder", B=4, K=8, N=211577, dtype="float32", L=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["gated", "gated", "clip", "beam", "reorder"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    if op == "gated":
        T = _log_int(rng, 1, 65_536)
        n = _log_int(rng, 2_000, 10_000_000)
        B = max(1, min(_log_int(rng, 1, 64), n // T // 4))
        return dict(op=op, T=T, B=B, N=max(1, min(20_000, n // (T * B))), dtype=dtype,
                    form=rng.choice(["leak", "decay"]), lengths=rng.random() < 0.4, grad=rng.random() < 0.7)
    if op == "clip":
        return dict(op=op, sizes=f"draw {rng.randrange(10 ** 6)} {_log_int(rng, 100, 1_000_000)}",
                    count=_log_int(rng, 1, 500), ratio=rng.choice([0.1, 0.5, 0.9, 2.0]),
                    mixed=rng.random() < 0.5)
    if op == "beam":
        V, K = _log_int(rng, 200, 131_072), rng.randint(1, 16)
        B = max(1, min(_log_int(rng, 1, 32), 30_000_000 // (V * K)))
        return dict(op=op, B=B, K=K, V=V, dtype=dtype, N=_log_int(rng, 64, 20_000), L=_log_int(rng, 8, 1024),
                    ended=rng.choice([0.0, 0.1, 0.4]))
    B, K = _log_int(rng, 1, 16), rng.randint(1, 16)
    return dict(op=op, B=B, K=K, N=_log_int(rng, 64, min(211_577, 6_000_000 // (B * K))), dtype=dtype,
                L=_log_int(rng, 8, 4096))


# -- inputs ----------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 104729 + 31)
    return g


def _tensors(c):
    """(elements, type) of each gradient."""
    kind = c["sizes"]
    if kind == "tiny":
        return [(4096, "float32"), (256, "float32"), (256, "float32")]
    if kind == "connectome":
        return [(24_678_466, "float32"), (211_577, "float32"), (211_577, "float32"),
                (256 * 211_577, "bfloat16")]
    rng = random.Random(kind)
    most = 400_000 if kind == "many" else int(kind.split()[2])
    sizes = [_log_int(rng, 1, most) for _ in range(c["count"])]
    return [(n, "bfloat16" if c["mixed"] and i % 2 else "float32") for i, n in enumerate(sizes)]


def _parents(B, K, g):
    """Beams that a step keeps: some twice, some not at all."""
    return torch.randint(0, K, (B, K), generator=g, device=_DEV)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    rand = lambda *n: torch.randn(*n, generator=g, device=_DEV)  # noqa: E731
    if c["op"] == "gated":
        T, B, N, dt = c["T"], c["B"], c["N"], _DT[c["dtype"]]
        if c["form"] == "leak":  # proposals in (-1, 1), leaks mostly between 0.02 and 0.9
            s["x"] = torch.tanh(rand(T, B, N)).to(dt)
            s["gate"] = (rand(T, B, N) * 1.5 - 1).to(dt)
        else:                    # decays mostly between 0.7 and 0.999
            s["x"] = (rand(T, B, N) * 0.1).to(dt)
            s["gate"] = torch.sigmoid(rand(T, B, N) * 1.5 + 3).to(dt)
        s["state0"] = torch.tanh(rand(B, N))
        s["lengths"] = None
        if c["lengths"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=g, device=_DEV)
        if c["grad"]:
            s["d_out"] = (rand(T, B, N) * 1e-2).to(dt)
            s["d_state"] = rand(B, N) * 1e-2
        return s
    if c["op"] == "clip":
        sizes = _tensors(c)
        s["grads"] = [(rand(n) * 1e-3).to(_DT[t]) for n, t in sizes]
        # where the clipped ones go: a line of memory for each type, a place of 16 bytes for each begin
        ends, s["flat"] = {}, {}
        at = []
        for n, t in sizes:
            at.append(ends.get(t, 0))
            ends[t] = at[-1] + -(-n // 8) * 8
        for t, n in ends.items():
            s["flat"][t] = torch.zeros(n, dtype=_DT[t], device=_DEV)
        s["out"] = [s["flat"][t][i:i + n] for i, (n, t) in zip(at, sizes)]
        s["max_norm"] = c["ratio"] * 1e-3 * math.sqrt(sum(n for n, _ in sizes))
        return s
    B, K, dt = c["B"], c["K"], _DT[c["dtype"]]
    if c["op"] == "reorder":
        s["parents"] = _parents(B, K, g)
        s["states"] = [torch.tanh(rand(B, K, c["N"])).to(dt),
                       torch.randint(0, 50_000, (B, K, c["L"]), generator=g, device=_DEV)]
        return s
    V = c["V"]
    s["logits"] = (rand(B, K, V) * 3).to(dt)
    s["scores"] = -torch.rand(B, K, generator=g, device=_DEV) * 10 - 20
    s["end_token"] = V // 3
    s["ended"] = None
    if c["ended"]:
        s["ended"] = torch.rand(B, K, generator=g, device=_DEV) < c["ended"]
    s["states"] = [torch.tanh(rand(B, K, c["N"])),
                   torch.randint(0, V, (B, K, c["L"]), generator=g, device=_DEV)]
    return s


# -- plain forms -----------------------------------------------------------------------------


def _scan(a, b):
    """h[t] = a[t] h[t - 1] + b[t] from h = 0, by doubling; overwrites both."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat((b[:d], a[d:] * b[:-d] + b[d:]))
        a = torch.cat((a[:d], a[d:] * a[:-d]))
        d *= 2
    return b


def _gated_plain(s):
    c = s["case"]
    T, B = c["T"], c["B"]
    x, f = s["x"].float(), s["gate"].float()
    if c["form"] == "leak":
        leak = 1 / (1 + torch.exp(-f))
        a, u = 1 / (1 + torch.exp(f)), leak * x
    else:
        a, u = f, x
    live = None
    if c["lengths"]:
        live = (torch.arange(T, device=_DEV).view(T, 1) < s["lengths"]).unsqueeze(-1)
        a, u = torch.where(live, a, 1.0), torch.where(live, u, 0.0)
    u = torch.cat((u[:1] + a[:1] * s["state0"], u[1:]))
    h = _scan(a, u)
    state = h[-1]
    out = {"out": (h if live is None else torch.where(live, h, 0.0)).to(s["x"].dtype), "state": state}
    if not c["grad"]:
        return out
    d = s["d_out"].float()
    if live is not None:
        d = torch.where(live, d, 0.0)
    d = torch.cat((d[:-1], d[-1:] + s["d_state"]))
    # g[t] = d[t] + a[t + 1] g[t + 1], read backwards
    later = torch.cat((a[1:], torch.zeros_like(a[:1])))
    grad = _scan(later.flip(0), d.flip(0)).flip(0)
    before = torch.cat((s["state0"].unsqueeze(0), h[:-1]))
    out["dstate0"] = a[0] * grad[0]
    if c["form"] == "leak":
        dx, dgate = grad * leak, grad * (x - before) * leak * (1 / (1 + torch.exp(f)))
    else:
        dx, dgate = grad, grad * before
    if live is not None:
        dx, dgate = torch.where(live, dx, 0.0), torch.where(live, dgate, 0.0)
    out["dx"], out["dgate"] = dx.to(s["x"].dtype), dgate.to(s["x"].dtype)
    return out


def _clip_plain(s):
    total = torch.zeros((), dtype=torch.float64, device=_DEV)
    for t in s["grads"]:
        v = t.float()
        total += (v * v).sum(dtype=torch.float64)
    norm = total.sqrt().float()
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * factor)
    return {"norm": norm, "grads": s["flat"]}


def _gather(states, parents):
    at = torch.arange(parents.shape[0], device=_DEV).unsqueeze(1)
    return [t[at, parents] for t in states]


def _beam_plain(s):
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    z = s["logits"].double()
    top = z.max(-1, keepdim=True).values
    total = top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))
    score = s["scores"].double().unsqueeze(-1) + (z - total)
    if s["ended"] is not None:
        only = torch.full((V,), -math.inf, dtype=torch.float64, device=_DEV)
        only[s["end_token"]] = 0.0
        stay = s["scores"].double().unsqueeze(-1) + only
        score = torch.where(s["ended"].unsqueeze(-1), stay, score)
    score = score.reshape(B, K * V)
    at = torch.arange(K * V, device=_DEV)
    best, where = [], []
    for _ in range(K):
        m = score.max(1, keepdim=True).values
        i = torch.where(score == m, at, K * V).min(1, keepdim=True).values
        best.append(m)
        where.append(i)
        score.scatter_(1, i, -math.inf)
    best, where = torch.cat(best, 1), torch.cat(where, 1)
    parents, tokens = where // V, where % V
    history = _gather(s["states"], parents)
    return {"scores": best.float(), "parents": parents, "tokens": tokens,
            "ended": tokens == s["end_token"], "states": history}


# -- one pass --------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "gated":
            return _gated_plain(s)
        if c["op"] == "clip":
            return _clip_plain(s)
        if c["op"] == "beam":
            return _beam_plain(s)
        return {"states": _gather(s["states"], s["parents"])}
    import sparse_graph_recurrent_gb300 as ck
    if c["op"] == "gated":
        args = dict(lengths=s["lengths"], form=c["form"])
        if not c["grad"]:
            out, state = ck.gated_recurrence(s["x"], s["gate"], s["state0"], **args)
            return {"out": out, "state": state}
        out, state, kept = ck.gated_recurrence_forward(s["x"], s["gate"], s["state0"], **args)
        dx, dgate, dstate0 = ck.gated_recurrence_backward(s["x"], s["gate"], kept, s["d_out"], s["d_state"],
                                                          **args)
        return {"out": out, "state": state, "dstate0": dstate0, "dx": dx, "dgate": dgate}
    if c["op"] == "clip":
        norm = ck.clip_gradients(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["flat"]}
    if c["op"] == "beam":
        scores, parents, tokens, ended = ck.beam_select(s["logits"], s["scores"], ended=s["ended"],
                                                        end_token=s["end_token"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "ended": ended,
                "states": ck.reorder_states(s["states"], parents)}
    return {"states": ck.reorder_states(s["states"], s["parents"])}


# -- what a pass cannot do without -----------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "gated":
        n, e, m = c["T"] * c["B"] * c["N"], _SIZE[c["dtype"]], c["B"] * c["N"]
        # x, gate in and states out; with gradients d_out in, two gradients out
        return {"bytes": n * e * (6 if c["grad"] else 3) + 4 * m * (4 if c["grad"] else 2),
                "flops": n * (20 if c["grad"] else 6)}
    if c["op"] == "clip":
        sizes = _tensors(c)
        return {"bytes": 2 * sum(n * _SIZE[t] for n, t in sizes) + 4, "flops": 3 * sum(n for n, _ in sizes)}
    B, K, N, L = c["B"], c["K"], c["N"], c["L"]
    if c["op"] == "reorder":
        return {"bytes": 2 * B * K * (N * _SIZE[c["dtype"]] + 8 * L) + 8 * B * K, "flops": B * K}
    n = B * K * c["V"]
    return {"bytes": n * _SIZE[c["dtype"]] + 2 * B * K * (4 * N + 8 * L) + 26 * B * K, "flops": 4 * n}


# -- the definitions in 64 bits --------------------------------------------------------------


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "gated":
        T = c["T"]
        x, f, h = s["x"].double(), s["gate"].double(), s["state0"].double()
        keep = 1 - torch.sigmoid(f) if c["form"] == "leak" else f
        enter = torch.sigmoid(f) if c["form"] == "leak" else torch.ones_like(f)
        put = enter * x
        inside = None
        if c["lengths"]:
            steps = torch.arange(T, device=_DEV).unsqueeze(1)
            inside = (s["lengths"].unsqueeze(0) > steps).unsqueeze(2).double()
            keep, put = keep * inside + (1 - inside), put * inside
        states = torch.empty(T + 1, *h.shape, dtype=torch.float64, device=_DEV)
        states[0] = h
        for t in range(T):
            torch.addcmul(put[t], keep[t], states[t], out=states[t + 1])
        got = {"out": states[1:] if inside is None else states[1:] * inside, "state": states[T]}
        if c["grad"]:
            d = s["d_out"].double()
            if inside is not None:
                d = d * inside
            g = torch.empty_like(states)
            g[T] = s["d_state"].double()
            total = torch.empty_like(d)
            for t in range(T - 1, -1, -1):
                torch.add(d[t], g[t + 1], out=total[t])
                torch.mul(keep[t], total[t], out=g[t])
            got["dstate0"] = g[0]
            if c["form"] == "leak":
                dx, dgate = total * enter, total * (x - states[:-1]) * enter * (1 - enter)
            else:
                dx, dgate = total, total * states[:-1]
            if inside is not None:
                dx, dgate = dx * inside, dgate * inside
            got["dx"], got["dgate"] = dx, dgate
        return got
    if c["op"] == "clip":
        parts = [t.double() for t in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(t, t)) for t in parts))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        lines = {}
        for t, part in zip(s["grads"], parts):
            gap = torch.zeros(-part.numel() % 8, dtype=torch.float64, device=_DEV)
            lines.setdefault(str(t.dtype).split(".")[1], []).extend((part * factor, gap))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": {k: torch.cat(v) for k, v in lines.items()}}
    if c["op"] == "reorder":
        rows = s["parents"].tolist()
        return {"states": [torch.stack([torch.stack([t[b, k] for k in r]) for b, r in enumerate(rows)])
                           for t in s["states"]]}
    B, K, V = c["B"], c["K"], c["V"]
    got = {k: [] for k in ("scores", "parents", "tokens")}
    for b in range(B):
        options = []
        for k in range(K):
            base = float(s["scores"][b, k])
            if s["ended"] is not None and bool(s["ended"][b, k]):
                options.append((-base, k, s["end_token"]))
                continue
            p = torch.log_softmax(s["logits"][b, k].double(), 0)
            v, i = torch.sort(p, descending=True, stable=True)
            options += [(-(base + w), k, j) for w, j in zip(v[:K].tolist(), i[:K].tolist())]
        options = sorted(options)[:K]
        got["scores"].append([-o[0] for o in options])
        got["parents"].append([o[1] for o in options])
        got["tokens"].append([o[2] for o in options])
    scores = torch.tensor(got["scores"], dtype=torch.float64)
    parents, tokens = torch.tensor(got["parents"]), torch.tensor(got["tokens"])
    kept = [torch.stack([t[b, parents[b].to(t.device)] for b in range(B)]) for t in s["states"]]
    return {"scores": scores, "parents": parents, "tokens": tokens, "ended": tokens == s["end_token"],
            "states": kept}
