"""Plain numpy definitions, in 64 bits, of the readout operators: the generator,
dropout, 4-bit weights and logit controls.  Test infrastructure only; shares
nothing with the library."""
import numpy as np

M32 = 0xFFFFFFFF


def philox_words(index, seed, step):
    """The generator's word for each element index (any integer array)."""
    index = np.asarray(index, dtype=np.uint64)
    u = np.uint64
    blk, lane = index >> u(2), (index & u(3)).astype(np.int64)
    c0, c1 = blk & u(M32), blk >> u(32)
    c2 = np.full_like(blk, int(step) & M32)
    c3 = np.full_like(blk, (int(step) >> 32) & M32)
    k0, k1 = int(seed) & M32, (int(seed) >> 32) & M32
    for _ in range(10):
        lo0, lo1 = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = ((lo1 >> u(32)) ^ c1 ^ u(k0), lo1 & u(M32),
                          (lo0 >> u(32)) ^ c3 ^ u(k1), lo0 & u(M32))
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return np.choose(lane, [c0, c1, c2, c3])


def keep_mask(shape, p, seed, step, locked):
    n = int(np.prod(shape[1:] if locked else shape))
    w = philox_words(np.arange(n), seed, step).astype(np.int64)
    keep = w >= int(np.rint(p * 2.0 ** 32))
    return np.broadcast_to(keep.reshape((1, *shape[1:]) if locked else shape), shape)


def unpack(q, K):
    """Nibbles [V, K] of packed rows [V, (K + 1) // 2]."""
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.int64)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out[:, :K]


def dequantize(q, scales, zeros, K, group):
    g = np.arange(K) // group
    z = 8 if zeros is None else (zeros.astype(np.int64) & 15)[:, g]
    return (unpack(q, K) - z) * scales.astype(np.float64)[:, g]


def controlled(logits, history=None, history_len=None, prompt_len=None, repetition=1.0,
               frequency=0.0, presence=0.0, bias=None, mask=None, temperature=1.0):
    """Controlled logits [B, V] in float64, one scalar at a time."""
    B, V = logits.shape
    z = logits.astype(np.float64).copy()
    per = lambda v, b: float(v[b]) if np.ndim(v) else float(v)  # noqa: E731
    for b in range(B):
        L = 0 if history is None else history.shape[1]
        n_used = L if history_len is None else min(max(int(history_len[b]), 0), L)
        n_prompt = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), L)
        seen, count = set(), {}
        for i in range(n_used):
            v = int(history[b, i])
            if not 0 <= v < V:
                continue
            seen.add(v)
            if i >= n_prompt:
                count[v] = count.get(v, 0) + 1
        r, f, pr, t = (per(v, b) for v in (repetition, frequency, presence, temperature))
        for v in seen:
            z[b, v] = z[b, v] / r if z[b, v] > 0 else z[b, v] * r
            if count.get(v, 0):
                z[b, v] -= count[v] * f + pr
        if bias is not None:
            z[b] += bias if bias.ndim == 1 else bias[b]
        if mask is not None:
            words = mask if mask.ndim == 1 else mask[b]
            for v in range(V):
                if not (int(words[v // 32]) >> (v % 32)) & 1:
                    z[b, v] = -np.inf
        if t > 0:
            z[b] /= t
    return z


def gumbel(B, V, seed, step):
    w = philox_words(np.arange(B * V), seed, step).astype(np.float64).reshape(B, V)
    u = np.minimum(w * 2.0 ** -32 + 2.0 ** -33, 1 - 2.0 ** -24)
    return -np.log(-np.log1p(-u))


def pick(score):
    out = []
    for row in score:
        s = np.where(np.isnan(row), -np.inf, row)
        out.append(int(np.argmax(s)) if (s > -np.inf).any() else -1)
    return np.array(out)
