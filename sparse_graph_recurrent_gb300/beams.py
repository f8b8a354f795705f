"""A step of beam search: which beams and tokens go on, and the beams' states moved to
their places.

    scores, parents, tokens, ended = beam_select(logits, scores, ended, end_token)
    state, history = reorder_states([state, history], parents)

Every call enqueues its kernels on the current stream and returns without waiting.
"""
from __future__ import annotations

import torch

from . import _ck
from .readout import _refuse_derivatives, _written

__all__ = ["beam_select", "reorder_states"]

_beam_ws = {}  # workspace bytes by (dtype, B, K, V, beams): sizes only, no memory


def beam_select(logits, scores, ended=None, end_token=None, beams=None):
    """The `beams` best (as many as there are, by default) of the K V candidates of each
    sequence: (scores, parents, tokens, ended), float32, int64, int64 and bool [B, beams],
    best first.  logits [B, K, V] (float32, bfloat16 or float16; after control_logits, where
    there are controls), scores float32 [B, K].  The score of beam k with token v is
    scores[b, k] + log_softmax(logits[b, k])[v]; of equal ones the lowest k, then the lowest v
    comes first.  The softmax's sum is one of 32-bit exponentials, whose logarithm is off by
    6e-6 at most (for 131,072 tokens), the rest is of 64 bits: candidates of one beam are in the
    order of their logits, those of different beams that lie closer than that may be taken in
    either order.  A beam with ended[b, k] (bool) goes on as one
    candidate, end_token at the score that it has; the ended that is returned says which
    beams are at end_token now.  A token at -inf or NaN is no candidate, nor is any of a
    beam whose score is not finite (the beams of a first step but one) or whose logits hold
    +inf.  Where candidates run out: score -inf, token -1, parent the beam of that place
    (0 past the last)."""
    got = (_ck._native or _ck.native()).beam(logits, scores, ended, end_token, beams)
    if got is not None:
        return got
    if not logits.is_cuda or logits.dtype not in _ck.DTYPES or logits.dim() != 3:
        raise ValueError("logits must be a CUDA tensor [B, K, V] of float32, bfloat16 or float16")
    _refuse_derivatives("beam_select", logits=logits, scores=scores)
    device, (B, K, V) = logits.get_device(), logits.shape
    beams = K if beams is None else int(beams)
    logits = logits.resolve_neg()
    if V > 1 and logits.stride(2) != 1:
        logits = logits.contiguous()
    _ck._like(scores, device, torch.float32, (B, K), "scores")
    scores = scores.resolve_neg().contiguous()
    if ended is not None:
        _ck._like(ended, device, torch.bool, (B, K), "ended")
        if end_token is None:
            raise ValueError("ended needs an end_token")
        ended = ended.contiguous()
    if end_token is not None and not 0 <= end_token < V:
        raise ValueError(f"end_token {end_token} is no token of {V}")
    key = (device, logits.dtype, B, K, V, beams)
    need = _beam_ws.get(key)
    if need is None:
        if len(_beam_ws) > 4096:
            _beam_ws.clear()
        with torch.cuda.device(device):
            need = _beam_ws[key] = _ck.ck_beam_workspace_size(logits.dtype, B, K, V, beams)
    new = lambda dtype: torch.empty((B, beams), dtype=dtype, device=logits.device)  # noqa: E731
    out = new(torch.float32), new(torch.int64), new(torch.int64), new(torch.bool)
    ws = torch.empty((need + 7) // 8, dtype=torch.int64, device=logits.device)
    call = _ck.BeamCall(logits.data_ptr(), _ck.DTYPES[logits.dtype], B, K, V, logits.stride(0), logits.stride(1),
                        scores.data_ptr(), None if ended is None else ended.data_ptr(),
                        -1 if end_token is None else int(end_token), beams, *(t.data_ptr() for t in out),
                        ws.data_ptr(), ws.numel() * 8)
    if device == _ck._get_device():
        _ck.ck_beam_select(call)
    else:
        with torch.cuda.device(device):
            _ck.ck_beam_select(call)
    return out


def _rows_inside(t):
    """Whether t[b, k] is a dense row, and strides are not negative."""
    at = 1
    for n, s in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        if n != 1 and s != at:
            return False
        at *= n
    return True


def _noted(t):
    """Whether t's numbers are the conjugated, the negated ones of what its memory holds."""
    return t.is_conj(), t.is_neg()


def reorder_states(states, parents, out=None):
    """states[b, parents[b, j]] for every sequence b and place j: new tensors
    [B, beams, ...] of a tensor [B, K, ...] or of several, of any types, in one pass.
    parents is int64 [B, beams] as beam_select returns it; one outside [0, K) gives zeros.
    `out`, a tensor or as many as there are states, is written instead; a state may be its
    own `out`, where beams == K.  An `out` that overlaps another array, or parents, is refused."""
    got = (_ck._native or _ck.native()).reorder(states, parents, out)
    if got is not None:
        return got
    single = isinstance(states, torch.Tensor)
    some = [states] if single else list(states)
    if parents.dtype != torch.int64 or parents.dim() != 2 or not parents.is_cuda:
        raise ValueError("parents must be a CUDA int64 tensor [B, beams]")
    device, (B, beams) = parents.get_device(), parents.shape
    parents = parents.contiguous()
    to = None if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    if to is not None and (len(to) != len(some) or single != isinstance(out, torch.Tensor)):
        raise ValueError("out holds as many tensors as there are states")
    if not some:
        return []
    K = some[0].shape[1] if some[0].dim() > 1 else 0
    array, held, result = (_ck.BeamState * len(some))(), [], []
    for i, (t, entry) in enumerate(zip(some, array)):
        if t.get_device() != device or t.dim() < 2 or t.shape[0] != B or t.shape[1] != K or t.layout != torch.strided:
            raise ValueError(f"a state must be a tensor [{B}, {K}, ...] on cuda:{device}, not {tuple(t.shape)} on {t.device}")
        _refuse_derivatives("reorder_states", state=t)
        if to is None:
            o = torch.empty((B, beams, *t.shape[2:]), dtype=t.dtype, device=t.device)
        else:
            o = to[i]
            if o.dtype != t.dtype or o.shape != (B, beams, *t.shape[2:]) or o.device != t.device:
                raise ValueError("out is like the states, [B, beams, ...]")
            _refuse_derivatives("reorder_states", out=o)
            if not _rows_inside(o):
                raise ValueError("the rows out[b, j] must be dense")
        source = t.detach()
        if not _rows_inside(source):
            source = source.contiguous()
        if _noted(source) != _noted(o):  # (alike, the bytes move as they are)
            source = source.resolve_conj().resolve_neg()
            if any(_noted(o)):
                raise ValueError("out is conjugated or negated lazily, and the state is not")
        size = t.element_size()
        entry.in_, entry.out, entry.bytes = source.data_ptr(), o.data_ptr(), source[0, 0].numel() * size if B and K else 0
        entry.in_row, entry.in_beam = source.stride(0) * size, source.stride(1) * size
        entry.out_row, entry.out_beam = o.stride(0) * size, o.stride(1) * size
        held.append(source)
        result.append(o)
    with torch.cuda.device(device):
        _ck.ck_reorder_states(array, parents, B, K, beams)
    if to is not None:
        for o in result:
            _written(o)
    return result[0] if single else result
