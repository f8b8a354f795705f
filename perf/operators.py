"""The readout operators at the sizes they are used at: counter-based dropout on
the recurrence's states, the product of states with a 4-bit readout, and the
controls that turn its logits into a token.

Each case runs either in plain form (elementary torch operations in 32 bits,
`own = False`) or through this framework's entry points (`own = True`).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
_DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # -- dropout of the states [T, B, N], forward and gradient ------------------------------
        # the tiny workload's window: one short training step, where the calls' latency counts
        dict(name="dropout_tiny", op="dropout", T=8, B=8, N=256, dtype="float32", p=0.1,
             locked=False, pad=0, grad=True),
        # the FlyGPT window, one mask for all 64 input steps
        dict(name="dropout_flygpt_locked", op="dropout", T=64, B=32, N=5000, dtype="float32",
             p=0.2, locked=True, pad=0, grad=True),
        # the ragged workload's batch of 20, odd node count, rows cut out of a wider buffer
        dict(name="dropout_ragged_half", op="dropout", T=32, B=20, N=4999, dtype="float16",
             p=0.5, locked=False, pad=9, grad=True),
        # the wide workload's states kept in bf16: the largest
        dict(name="dropout_wide_bf16", op="dropout", T=32, B=256, N=20000, dtype="bfloat16",
             p=0.1, locked=False, pad=0, grad=False),
        # -- the 4-bit readout ------------------------------------------------------------------
        # one byte-level sequence being answered: 256 logits from 5,000 node states
        dict(name="readout_bytes_1", op="int4", M=1, K=5000, V=256, group=64, dtype="float32",
             zeros=False, bias=True),
        # the FlyGPT batch of 32 sequences, a vocabulary of words, the framework's own fp32 states
        dict(name="readout_words_32", op="int4", M=32, K=5000, V=32000, group=128,
             dtype="float32", zeros=False, bias=False),
        # four sequences over the wide workload's nodes, short groups with zero points
        dict(name="readout_wide_4", op="int4", M=4, K=20000, V=16384, group=32, dtype="float16",
             zeros=True, bias=False),
        # one sequence over the whole connectome: the long axis, an odd number of nodes
        dict(name="readout_connectome_1", op="int4", M=1, K=211577, V=4096, group=128,
             dtype="bfloat16", zeros=True, bias=True),
        # -- controls on logits, and the token --------------------------------------------------
        # one byte-level sequence, greedy: the smallest call of an answering loop
        dict(name="token_bytes_1", op="logits", B=1, V=256, L=64, dtype="float32", mask=0.5,
             bias="row", pick="greedy", logits_out=False, prompt=0.5),
        # 32 sequences sampled under a grammar that leaves few tokens; only tokens are wanted
        dict(name="token_words_32", op="logits", B=32, V=32000, L=1024, dtype="float32",
             mask=0.05, bias="none", pick="sample", logits_out=False, prompt=0.25),
        # controls alone, odd vocabulary, long histories, a bias of its own for each row
        dict(name="control_ragged_20", op="logits", B=20, V=50021, L=32768, dtype="float16",
             mask=0.0, bias="rows", pick="none", logits_out=True, prompt=0.9),
        # a large vocabulary at a large batch, sampled, the controlled logits wanted too
        dict(name="token_large_64", op="logits", B=64, V=131072, L=4096, dtype="bfloat16",
             mask=0.3, bias="row", pick="sample", logits_out=True, prompt=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    op = rng.choice(["dropout", "int4", "logits"])
    if op == "dropout":
        n = _log_int(rng, 16_000, 160_000_000 if dtype != "float32" else 60_000_000)
        T = rng.randint(1, 64)
        B = max(1, min(_log_int(rng, 1, 256), n // T // 8))
        N = max(1, n // (T * B))
        grad = rng.random() < 0.6
        return dict(op=op, T=T, B=B, N=max(1, N // 2 if grad else N), dtype=dtype,
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]), locked=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 3, 16]), grad=grad)
    if op == "int4":
        K = _log_int(rng, 256, 211_577)
        V = _log_int(rng, 200, min(64_000, max(400, 860_000_000 // K)))
        M = max(1, min(_log_int(rng, 1, 32), 5_000_000_000 // (K * V)))
        return dict(op=op, M=M, K=K, V=V, group=rng.choice([32, 64, 128]), dtype=dtype,
                    zeros=rng.random() < 0.5, bias=rng.random() < 0.5)
    V = _log_int(rng, 200, 262_144)
    B = min(_log_int(rng, 1, 128), max(1, 8_000_000 // V))
    pick = rng.choice(["none", "greedy", "sample", "sample"])
    return dict(op=op, B=B, V=V, L=_log_int(rng, 16, 32_768), dtype=dtype,
                mask=rng.choice([0.0, 0.05, 0.5]), bias=rng.choice(["none", "row", "rows"]),
                pick=pick, logits_out=pick == "none" or rng.random() < 0.5,
                prompt=rng.choice([0.0, 0.3, 0.8]))


# -- inputs ----------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _groups(c):
    return -(-c["K"] // c["group"])


def _pitch(K):
    """Bytes between rows of packed weights: K nibbles, to a multiple of 16 bytes."""
    return -(-((K + 1) // 2) // 16) * 16


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dt = _DT[c["dtype"]]
    s = {"case": c}
    if c["op"] == "dropout":
        # states of the leaky-tanh recurrence lie in (-1, 1); their gradients are small
        shape = (c["T"], c["B"], c["N"] + c["pad"])
        x = torch.tanh(torch.randn(shape, generator=g, device=_DEV)).to(dt)
        s["x"] = x[..., :c["N"]]
        if c["grad"]:
            d = (torch.randn(shape, generator=g, device=_DEV) * 1e-2).to(dt)
            s["d"] = d[..., :c["N"]]
        s["seed"], s["step"] = 0x9E3779B97F4A7C15 ^ (int(seed) * 2654435761), int(seed) % 100_003
        return s
    if c["op"] == "int4":
        M, K, V, G = c["M"], c["K"], c["V"], _groups(c)
        s["x"] = torch.tanh(torch.randn(M, K, generator=g, device=_DEV)).to(dt)
        # nibbles as rounding normal weights leaves them: two draws per byte around 8
        b = torch.empty(V, _pitch(K), dtype=torch.uint8, device=_DEV)
        for r in range(0, V, 8192):
            part = b[r:r + 8192]
            lo = torch.randn(part.shape, generator=g, device=_DEV).mul_(2.6).add_(8).round_().clamp_(0, 15)
            hi = torch.randn(part.shape, generator=g, device=_DEV).mul_(2.6).add_(8).round_().clamp_(0, 15)
            part.copy_(lo + 16 * hi)
        s["qweight"] = b[:, :(K + 1) // 2]
        s["scales"] = ((0.5 + torch.rand(V, G, generator=g, device=_DEV)) * (0.4 / math.sqrt(K))).to(dt)
        s["zeros"] = (torch.randint(5, 12, (V, G), generator=g, device=_DEV).to(torch.uint8)
                      if c["zeros"] else None)
        s["bias"] = torch.randn(V, generator=g, device=_DEV) if c["bias"] else None
        return s
    B, V, L = c["B"], c["V"], c["L"]
    s["logits"] = (torch.randn(B, V, generator=g, device=_DEV) * 3).to(dt)
    # token ids of text: a few are frequent, most are rare
    u = torch.rand(B, L, generator=g, device=_DEV)
    s["history"] = (V * u.pow(4)).long().clamp_(max=V - 1)
    s["history_len"] = torch.randint(max(1, L // 2), L + 1, (B,), generator=g, device=_DEV)
    s["prompt_len"] = (s["history_len"] * c["prompt"]).long()
    s["repetition"] = 1.0 + 0.5 * torch.rand(B, generator=g, device=_DEV)
    s["frequency"] = 0.3 * torch.rand(B, generator=g, device=_DEV)
    s["presence"] = 0.5 * torch.rand(B, generator=g, device=_DEV)
    s["temperature"] = 0.6 + torch.rand(B, generator=g, device=_DEV)
    s["bias"] = None
    if c["bias"] != "none":
        shape = (V,) if c["bias"] == "row" else (B, V)
        s["bias"] = torch.randn(shape, generator=g, device=_DEV) * (
            torch.rand(shape, generator=g, device=_DEV) < 0.02)
    s["mask"] = None
    if c["mask"]:
        W = -(-V // 32)
        bits = torch.rand(B, W, 32, generator=g, device=_DEV) < c["mask"]
        w = (bits.long() << torch.arange(32, device=_DEV)).sum(-1)
        s["mask"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    s["seed"] = (int(seed) * 0x2545F4914F6CDD1D + 12345) % 2 ** 63 if c["pick"] == "sample" else None
    s["step"] = int(seed) % 9973
    return s


# -- plain forms -----------------------------------------------------------------------------


def _words(n, seed, step):
    """The first n 32-bit words of the generator (Philox-4x32-10), as int64."""
    low = 0xFFFFFFFF
    blk = torch.arange(-(-n // 4), device=_DEV)
    a, b = blk & low, blk >> 32
    c, d = torch.full_like(blk, step & low), torch.full_like(blk, (step >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((y >> 32) & low) ^ b ^ k0, y & low, ((x >> 32) & low) ^ d ^ k1, x & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((a, b, c, d), -1).reshape(-1)[:n]


def _dropout_plain(xs, c, seed, step):
    shape = (1, c["B"], c["N"]) if c["locked"] else (c["T"], c["B"], c["N"])
    keep = (_words(math.prod(shape), seed, step) >= round(c["p"] * 2 ** 32)).view(shape)
    scale = torch.tensor(1.0 / (1.0 - c["p"]), dtype=torch.float32, device=_DEV)
    return [torch.where(keep, x.float() * scale, 0.0).to(x.dtype) for x in xs]


def _int4_plain(s):
    c = s["case"]
    K, V, G, n = c["K"], c["V"], _groups(c), c["group"]
    b = s["qweight"]
    q = torch.stack((b & 15, b >> 4), -1).view(V, -1)[:, :K]
    z = s["zeros"].float() if c["zeros"] else torch.full((V, G), 8.0, device=_DEV)
    at = torch.arange(K, device=_DEV) // n
    w = (q.float() - z[:, at]) * s["scales"].float()[:, at]
    y = s["x"].float() @ w.t()
    if c["bias"]:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _logits_plain(s):
    c = s["case"]
    B, V, L = c["B"], c["V"], c["L"]
    z = s["logits"].float()
    col = lambda v: v.view(B, 1)  # noqa: E731
    pos = torch.arange(L, device=_DEV).view(1, L)
    used = pos < col(s["history_len"])
    made = used & (pos >= col(s["prompt_len"]))
    seen = torch.zeros(B, V, dtype=torch.int32, device=_DEV)
    seen.scatter_add_(1, s["history"], used.int())
    count = torch.zeros(B, V, dtype=torch.int32, device=_DEV)
    count.scatter_add_(1, s["history"], made.int())
    r = col(s["repetition"])
    z = torch.where(seen > 0, torch.where(z > 0, z / r, z * r), z)
    z = z - (count.float() * col(s["frequency"]) + (count > 0).float() * col(s["presence"]))
    if s["bias"] is not None:
        z = z + s["bias"]
    if s["mask"] is not None:
        bits = (s["mask"].view(B, -1, 1) >> torch.arange(32, device=_DEV, dtype=torch.int32)) & 1
        z = torch.where(bits.view(B, -1)[:, :V] > 0, z, -math.inf)
    z = z / col(s["temperature"])
    out = {}
    if c["logits_out"]:
        out["logits"] = z.to(s["logits"].dtype)
    if c["pick"] != "none":
        score = z
        if c["pick"] == "sample":
            u = _words(B * V, s["seed"], s["step"]).float() * 2.0 ** -32 + 2.0 ** -33
            u = u.clamp(max=1 - 2.0 ** -24).view(B, V)
            score = z - torch.log(-torch.log1p(-u))
        best = score.max(1, keepdim=True).values
        first = torch.where(score == best, torch.arange(V, device=_DEV), V).min(1).values
        out["tokens"] = torch.where(best.view(B) > -math.inf, first, -1)
    return out


# -- one pass --------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "dropout":
            y = _dropout_plain([s["x"], s["d"]] if c["grad"] else [s["x"]], c, s["seed"], s["step"])
            return dict(zip(("y", "dx"), y))
        if c["op"] == "int4":
            return _int4_plain(s)
        return _logits_plain(s)
    import sparse_graph_recurrent_gb300 as ck
    if c["op"] == "dropout":
        out = {"y": ck.dropout(s["x"], c["p"], s["seed"], s["step"], locked=c["locked"])}
        if c["grad"]:
            out["dx"] = ck.dropout_backward(s["d"], c["p"], s["seed"], s["step"], locked=c["locked"])
        return out
    if c["op"] == "int4":
        return ck.int4_matvec(s["x"], s["qweight"], s["scales"], zeros=s["zeros"], bias=s["bias"],
                              group_size=c["group"])
    args = dict(history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"],
                repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                bias=s["bias"], mask=s["mask"], temperature=s["temperature"])
    if c["pick"] == "none":
        return {"logits": ck.control_logits(s["logits"], **args)}
    got = ck.pick_tokens(s["logits"], **args, seed=s["seed"], step=s["step"],
                         return_logits=c["logits_out"])
    return {"tokens": got[0], "logits": got[1]} if c["logits_out"] else {"tokens": got}


# -- what a pass cannot do without -----------------------------------------------------------


def work(case):
    c = case
    e = _SIZE[c["dtype"]]
    if c["op"] == "dropout":
        n = c["T"] * c["B"] * c["N"] * (2 if c["grad"] else 1)
        return {"bytes": 2 * n * e, "flops": n}
    if c["op"] == "int4":
        M, K, V, G = c["M"], c["K"], c["V"], _groups(c)
        b = V * ((K + 1) // 2) + V * G * (e + int(c["zeros"])) + (M * K + M * V) * e
        return {"bytes": b + 4 * V * int(c["bias"]), "flops": 2 * M * K * V}
    B, V = c["B"], c["V"]
    # token ids of 8 bytes, three quarters of the history used on average
    b = B * V * e * (2 if c["logits_out"] else 1) + 6 * B * c["L"] + 40 * B
    b += {"none": 0, "row": 4 * V, "rows": 4 * B * V}[c["bias"]]
    b += B * -(-V // 32) * 4 if c["mask"] else 0
    return {"bytes": b, "flops": B * V * (12 if c["pick"] == "sample" else 4)}


# -- the definitions in 64 bits --------------------------------------------------------------


def _exact_words(index, seed, step):
    """Words of the generator at the element indexes given (uint64 arrays on the host)."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    block, lane = index // u(4), index % u(4)
    ctr = [block & low, block >> u(32), np.full_like(block, step & 0xFFFFFFFF),
           np.full_like(block, step >> 32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        p0, p1 = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(p1 >> u(32)) ^ ctr[1] ^ u((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), p1 & low,
               (p0 >> u(32)) ^ ctr[3] ^ u((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF), p0 & low]
    return np.choose(lane.astype(np.int64), ctr)


def exact(case, seed):
    c = dict(case)
    if c["op"] == "dropout":
        n = (1 if c["locked"] else c["T"]) * c["B"] * c["N"]
        if n * (2 if c["grad"] else 1) > 20_000_000 or c["T"] * c["B"] * c["N"] > 30_000_000:
            return None
        s = prepare(case, seed)
        word = _exact_words(np.arange(n, dtype=np.uint64), s["seed"], s["step"])
        keep = (word.astype(np.float64) >= np.rint(c["p"] * 2.0 ** 32)).reshape(-1, c["B"], c["N"])
        out = {}
        for name, key in (("y", "x"), ("dx", "d")):
            if key in s:
                v = s[key].double().cpu().numpy()
                out[name] = np.where(keep, v / (1.0 - c["p"]), 0.0)
        return out
    s = prepare(case, seed)
    if c["op"] == "int4":
        M, K, V, n = c["M"], c["K"], c["V"], c["group"]
        x = s["x"].double()
        k = torch.arange(K, device=_DEV)
        y = torch.zeros(M, V, dtype=torch.float64, device=_DEV)
        rows = max(1, 100_000_000 // K)
        for r in range(0, V, rows):
            q = (s["qweight"][r:r + rows].int()[:, k // 2] >> (4 * (k % 2)).int()) % 16
            part = torch.zeros(q.shape[0], _groups(c) * n, dtype=torch.float64, device=_DEV)
            part[:, :K] = q
            part = part.view(q.shape[0], -1, n)
            part = part - (s["zeros"][r:r + rows].double().unsqueeze(-1) if c["zeros"] else 8.0)
            part = part * s["scales"][r:r + rows].double().unsqueeze(-1)
            y[:, r:r + rows] = torch.einsum("mk,vk->mv", x, part.view(q.shape[0], -1)[:, :K])
        if c["bias"]:
            y += s["bias"].double()
        return y
    B, V = c["B"], c["V"]
    host = {k: v.cpu().numpy() if v.dtype != torch.bfloat16 else v.float().cpu().numpy()
            for k, v in s.items() if isinstance(v, torch.Tensor)}
    z = host["logits"].astype(np.float64)
    tokens = np.full(B, -1, np.int64)
    for b in range(B):
        text = host["history"][b, :host["history_len"][b]]
        n = np.bincount(text[host["prompt_len"][b]:], minlength=V)
        old, row, r = np.unique(text), z[b], float(host["repetition"][b])
        row[old] = np.where(row[old] > 0, row[old] / r, row[old] * r)
        row -= n * float(host["frequency"][b])
        row[n > 0] -= float(host["presence"][b])
        if s["bias"] is not None:
            row += host["bias"] if c["bias"] == "row" else host["bias"][b]
        if s["mask"] is not None:
            bits = np.unpackbits(host["mask"][b].view(np.uint8), bitorder="little")[:V]
            row[bits == 0] = -np.inf
        row /= float(host["temperature"][b])
        if c["pick"] != "none":
            score = row.copy()
            if c["pick"] == "sample":
                at = np.arange(b * V, (b + 1) * V, dtype=np.uint64)
                u = (_exact_words(at, s["seed"], s["step"]) + 0.5) * 2.0 ** -32
                score -= np.log(-np.log1p(-np.minimum(u, 1 - 2.0 ** -24)))
            tokens[b] = int(np.argmax(score)) if np.isfinite(score).any() else -1
    out = {"logits": z} if c["logits_out"] else {}
    if c["pick"] != "none":
        out["tokens"] = tokens
    return out
