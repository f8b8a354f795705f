"""Plain numpy definitions, in 64 bits, of the gated recurrence, of clipping and of a beam
search's step, with bounds of what 32-bit arithmetic may be off by.  Test infrastructure
only; shares nothing with the library."""
import numpy as np

U32 = 2.0 ** -24  # half a step of a 32-bit float, relative


def _gates(x, gate, form):
    """What a step keeps of the state, what it puts in, and the leak."""
    if form == "leak":
        with np.errstate(over="ignore"):
            leak = 1 / (1 + np.exp(-gate))
            return 1 / (1 + np.exp(gate)), leak * x, leak
    return gate, x, None


def gated(x, gate, state0, lengths, form, d_out=None, d_state=None):
    """The recurrence over [T, B, N] and, given d_out, its gradients: a dict of values and a
    dict of bounds.

    A bound: each step multiplies and adds once, on numbers that are themselves rounded.  A
    term of h_t that entered j steps ago has at most C (j + 1) relative half steps of error,
    whatever the order in which the maps are composed, with C = 12: the gate (a sigmoid from
    an exponential of 2 units and a quotient, 8 half steps), its product with the running
    product or state, the sum, and one more each for a composition.  So with G the sum of the
    terms' absolute values and D that of (j + 1) times them the error is at most C U32 D."""
    C = 12 * U32
    T, B, N = x.shape
    live = np.ones((T, B, 1), bool) if lengths is None else (np.arange(T)[:, None] < lengths)[..., None]
    live = np.broadcast_to(live, x.shape)
    x, gate = np.where(live, x, 0.0), np.where(live, gate, 0.0)
    a, u, leak = _gates(x, gate, form)
    a, u = np.where(live, a, 1.0), np.where(live, u, 0.0)
    h = np.zeros((T + 1, B, N)) if state0 is None else np.concatenate((state0[None], np.zeros((T, B, N))))
    G, D = np.abs(h), np.zeros_like(h)
    for t in range(T):
        h[t + 1] = a[t] * h[t] + u[t]
        G[t + 1] = np.abs(a[t]) * G[t] + np.abs(u[t])
        D[t + 1] = np.abs(a[t]) * D[t] + np.where(live[t], G[t + 1], 0)
    got = {"out": np.where(live, h[1:], 0.0), "state": h[T]}
    off = {"out": np.where(live, C * D[1:], 0.0), "state": C * D[T]}
    if d_out is None:
        return got, off
    d = np.where(live, d_out, 0.0)
    r, RG, RD = np.zeros_like(h), np.zeros_like(h), np.zeros_like(h)
    g, gd = np.zeros_like(x), np.zeros_like(x)
    if d_state is not None:
        r[T] = d_state
        RG[T] = np.abs(d_state)
    for t in range(T - 1, -1, -1):
        g[t] = d[t] + r[t + 1]
        gg = np.abs(d[t]) + RG[t + 1]
        gd[t] = RD[t + 1] + gg
        r[t] = a[t] * g[t]
        RG[t] = np.abs(a[t]) * gg
        RD[t] = np.where(live[t], np.abs(a[t]) * gd[t] + RG[t], RD[t + 1])
        RG[t] = np.where(live[t], RG[t], RG[t + 1])
        r[t] = np.where(live[t], r[t], r[t + 1])
    got["dstate0"], off["dstate0"] = r[0], C * RD[0]
    err = C * gd
    before, before_off = h[:-1], C * D[:-1]
    if form == "leak":
        w = x - before
        got["dx"], off["dx"] = g * leak, err * leak + C * np.abs(g * leak)
        f = leak * a
        got["dgate"] = g * w * f
        off["dgate"] = f * (np.abs(w) * err + (np.abs(g) + err) * (before_off + U32 * np.abs(w))) + C * np.abs(g * w * f)
    else:
        got["dx"], off["dx"] = g, err
        got["dgate"] = g * before
        off["dgate"] = np.abs(before) * err + (np.abs(g) + err) * before_off + C * np.abs(g * before)
    for k in ("dx", "dgate"):
        got[k], off[k] = np.where(live, got[k], 0.0), np.where(live, off[k], 0.0)
    return got, off


def half_step(dtype):
    """(relative, absolute) half a step of a type named like torch's."""
    return {"float32": (2.0 ** -24, 2.0 ** -149), "bfloat16": (2.0 ** -8, 2.0 ** -133),
            "float16": (2.0 ** -11, 2.0 ** -25)}[dtype]


def within(got, want, off, dtype="float32"):
    """Whether got, rounded once to dtype, lies within `off` of want before the rounding
    (twice the bound of 64 bits against itself is nothing beside it)."""
    got = np.asarray(got, np.float64)
    rel, least = half_step(dtype)
    tol = off + (np.abs(want) + off) * rel + least
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / tol, 0)), bad.shape)
        raise AssertionError(f"{bad.sum()} of {bad.size} off; at {i}: {got[i]} for {want[i]}, tolerance {tol[i]}")


def clip(grads, max_norm):
    """(norm, factor) of a list of arrays in 64 bits."""
    with np.errstate(over="ignore", invalid="ignore"):
        norm = np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads))
        f = max_norm / (norm + 1e-6)
    return norm, (1.0 if f >= 1 else f)


def beam(logits, scores, ended, end_token, beams):
    """(scores, parents, tokens, ended) of a step of beam search."""
    B, K, V = logits.shape
    out = np.full((B, beams), -np.inf), np.zeros((B, beams), np.int64), np.full((B, beams), -1), np.zeros((B, beams), bool)
    for b in range(B):
        options = []
        for k in range(K):
            z, s = logits[b, k].astype(np.float64), float(scores[b, k])
            if not np.isfinite(s):
                continue
            if ended is not None and ended[b, k]:
                options.append((-s, k, end_token))
                continue
            z = np.where(np.isnan(z), -np.inf, z)
            top = z.max()
            if not np.isfinite(top):
                continue
            lse = top + np.log(np.exp(z - top).sum())
            best = np.argsort(-z, kind="stable")[:beams]
            options += [(-(s - lse + z[v]), k, int(v)) for v in best if z[v] > -np.inf]
        options.sort()
        for j in range(beams):
            if j < len(options):
                out[0][b, j], out[1][b, j], out[2][b, j] = -options[j][0], options[j][1], options[j][2]
                out[3][b, j] = options[j][2] == end_token
            else:
                out[1][b, j] = j if j < K else 0
    return out


def beam_score_off(V):
    """What a score may be off by, before its rounding: a sum of 32-bit exponentials.  Each
    is off by 2 + 1.2 |x| units (the intrinsic's documented bound), |x| on average no more
    than log V + 1 over the sum; a thread adds 32 of them, the rest is in 64 bits."""
    return (36 + 1.2 * (np.log(V) + 1)) * 2.0 ** -23
