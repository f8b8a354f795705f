"""From the states of a recurrent token model to its next token: dropout on the
states while it trains, a 4-bit readout and the controls on its logits while it
answers (connectome-kernels page, intro: a connectome trained on text).

    h = dropout(out, 0.2, seed, step, locked=True)          # training, differentiable
    q, scales, zeros = int4_quantize(w_readout)              # once
    logits = int4_matvec(state, q, scales, zeros)            # [B, N] -> [B, V]
    tokens = pick_tokens(logits, history, history_len=n, repetition=1.1,
                         mask=allowed, temperature=0.8, seed=seed, step=step)

Every call enqueues its kernels on the current stream and returns without waiting.
A call whose arguments are all in order goes through the compiled module
ck_binding; what that leaves is done, or refused, here.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _ck

__all__ = ["dropout", "dropout_backward", "int4_quantize", "int4_rows", "int4_matvec", "control_logits",
           "pick_tokens"]


def _followed(t) -> bool:
    """Whether autograd follows t: it is to get a gradient, or carries a tangent."""
    return (t.requires_grad and torch.is_grad_enabled()
            or forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None)


def _refuse_derivatives(what, **operands):
    for name, t in operands.items():
        if isinstance(t, torch.Tensor) and _followed(t):
            raise ValueError(f"{what} has no derivative: call it under no_grad or on a detached {name}")


def _written(out):
    if not out.is_inference():  # those have no version
        increment_version(out)


# -- dropout ---------------------------------------------------------------------------------


def _as3(x, locked):
    """x as [n0][n1][n2] (with its first axis alone when locked): (x, sizes,
    strides); a copy where its axes do not join into that many."""
    if x.is_contiguous():
        n = x.numel()
        if not locked:
            return x, (1, 1, n), (0, 0, 1)
        n0 = x.shape[0]
        m = n // n0 if n0 else 0
        return x, (n0, 1, m), (m, 0, 1)
    dims = [(n, s) for n, s in zip(x.shape, x.stride())]
    head, dims = (dims[:1], dims[1:]) if locked else ([], dims)
    joined = []
    for n, s in dims:
        if n == 1:
            continue
        if joined and joined[-1][1] == s * n:
            joined[-1] = (joined[-1][0] * n, s)
        else:
            joined.append((n, s))
    if len(head) + len(joined) > 3:
        return _as3(x.contiguous(), locked)
    joined = [(1, 0)] * (3 - len(head) - len(joined)) + joined
    dims = head + joined
    return x, tuple(n for n, _ in dims), tuple(s for _, s in dims)


def _dropout(x, p, seed, step, locked):
    device = x.get_device()
    if device < 0:
        raise ValueError("dropout takes CUDA tensors")
    if locked and x.dim() < 2:
        raise ValueError("a locked mask is shared along the first of at least two dimensions")
    if x.is_contiguous():
        y = torch.empty_like(x)
    else:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    x, shape, strides = _as3(x, locked)
    if device == _ck._get_device():
        _ck.ck_dropout(x, y, *shape, *strides, p, seed, step, locked)
    else:
        with torch.cuda.device(device):
            _ck.ck_dropout(x, y, *shape, *strides, p, seed, step, locked)
    return y


class _Dropout(torch.autograd.Function):
    """A linear map and its own transpose: the gradient and the tangent are dropout again,
    differentiable in their turn."""

    @staticmethod
    def forward(ctx, x, p, seed, step, locked):
        if isinstance(step, torch.Tensor):
            step = step.clone()  # the backward's mask is this forward's, wherever the counter is by then
        ctx.args = (p, seed, step, locked)
        x = x.detach()
        y = (_ck._native or _ck.native()).dropout(x, *ctx.args)
        return _dropout(x, *ctx.args) if y is None else y

    @staticmethod
    def backward(ctx, d_out):
        return dropout(d_out, *ctx.args), None, None, None, None

    @staticmethod
    def jvp(ctx, x_tangent, *_):
        return dropout(x_tangent, *ctx.args)


def dropout(x, p: float, seed: int, step=0, locked: bool = False):
    """x with each element kept and scaled by 1 / (1 - p), or set to 0 with
    probability p, differentiable in x.  The mask follows from (seed, step) and
    an element's index and is stored nowhere; give every call of a program a
    seed of its own and every training step another `step`, an int or a device
    int64[1] that ck_step_advance counts up (also inside a captured step).
    With locked=True one mask serves every entry of the first dimension, as for
    the T input steps of out[T, B, N].  float32, bfloat16 or float16, any strides."""
    y = (_ck._native or _ck.native()).dropout(x, p, seed, step, locked)
    if y is not None:
        return y
    if _followed(x):
        return _Dropout.apply(x, p, seed, step, locked)
    return _dropout(x, p, seed, step, locked)


def dropout_backward(d_out, p: float, seed: int, step=0, locked: bool = False):
    """The gradient of dropout's x from its output's: the same mask and factor again, so
    differentiable in d_out as dropout is in x."""
    y = (_ck._native or _ck.native()).dropout(d_out, p, seed, step, locked)
    return dropout(d_out, p, seed, step, locked) if y is None else y


# -- the 4-bit readout -----------------------------------------------------------------------


def int4_quantize(w, group_size: int = 128, symmetric: bool = True, scale_dtype=None):
    """4-bit weights of w [V, K] in groups of 32, 64 or 128 along K: (qweight,
    scales, zeros) for int4_matvec, zeros None when symmetric.  qweight is uint8
    [V, (K + 1) // 2], low nibble first, its rows at a multiple of 16 bytes (see
    int4_rows); scales [V, ceil(K / group_size)] in scale_dtype (w's by default)."""
    if w.dim() != 2 or w.shape[1] < 1 or not w.is_cuda:
        raise ValueError("w must be a CUDA tensor [V, K] with K >= 1")
    if group_size not in _ck.INT4_GROUPS:
        raise ValueError(f"group_size must be one of {_ck.INT4_GROUPS}, not {group_size}")
    w = w.detach()
    if w.shape[1] > 1 and w.stride(1) != 1:
        w = w.contiguous()
    V, K = w.shape
    G, n = -(-K // group_size), (K + 1) // 2
    q = torch.zeros((V, -(-n // 16) * 16), dtype=torch.uint8, device=w.device)[:, :n]
    scales = torch.empty((V, G), dtype=scale_dtype or w.dtype, device=w.device)
    zeros = None if symmetric else torch.empty((V, G), dtype=torch.uint8, device=w.device)
    with torch.cuda.device(w.device):
        _ck.ck_int4_quantize(w, group_size, q, scales, zeros)
    return q, scales, zeros


def int4_rows(qweight):
    """qweight uint8 [V, (K + 1) // 2] with its rows at a multiple of 16 bytes, as the
    product reads them: itself, or a copy where clone, to or a concatenation has put
    the rows one after another."""
    if qweight.dim() != 2 or qweight.dtype != torch.uint8:
        raise ValueError("qweight must be uint8 [V, (K + 1) // 2]")
    V, n = qweight.shape
    if ((V < 2 or qweight.stride(0) % 16 == 0) and (n < 2 or qweight.stride(1) == 1)
            and qweight.data_ptr() % 16 == 0):
        return qweight
    q = torch.zeros((V, -(-n // 16) * 16), dtype=torch.uint8, device=qweight.device)[:, :n]
    return q.copy_(qweight)


def int4_matvec(x, qweight, scales, zeros=None, bias=None, group_size: int = 128, out=None):
    """x [..., K] times the transpose of the 4-bit weights (int4_quantize), plus
    bias (float32 [V]): [..., V] in x's type.  For a few rows of x at a time, as
    when answering; it has no gradient.  `out`, if given, is written instead of a
    new tensor.  Weights whose rows follow one another without a gap, and not at
    multiples of 16 bytes, are laid out by int4_rows in every call."""
    y = (_ck._native or _ck.native()).int4_matvec(x, qweight, scales, zeros, bias, group_size, out)
    if y is not None:
        return y
    _refuse_derivatives("int4_matvec", x=x, scales=scales, bias=bias, out=out)
    device = x.get_device()
    if device < 0:
        raise ValueError("int4_matvec takes CUDA tensors")
    if x.dim() < 1 or qweight.dim() != 2:
        raise ValueError("x is [..., K] and qweight [V, (K + 1) // 2]")
    V = qweight.shape[0]
    if V > 1 and qweight.shape[1] % 16 and qweight.dtype == torch.uint8 and qweight.is_contiguous():
        qweight = int4_rows(qweight)
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    if x2.shape[1] > 1 and x2.stride(1) != 1:
        x2 = x2.contiguous()
    if out is None:
        y = torch.empty((x2.shape[0], V), dtype=x.dtype, device=x.device)
    else:
        if tuple(out.shape) != (*x.shape[:-1], V):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(*x.shape[:-1], V)}")
        y = out if out.dim() == 2 else out.view(-1, V)
        _written(out)
    args = (x2, qweight, scales, zeros, bias, group_size, y)
    if device == _ck._get_device():
        _ck.ck_int4_matvec(*args)
    else:
        with torch.cuda.device(device):
            _ck.ck_int4_matvec(*args)
    if out is not None:
        return out
    return y if x.dim() == 2 else y.view(*x.shape[:-1], V)


# -- controls on logits, and the token -------------------------------------------------------


_MOST = 3.4028234663852886e38   # of 32-bit floats the largest
_LEAST = 1.401298464324817e-45  # and the smallest above 0


def _per_row(name, v, default, low, B, device):
    """(pointer, number) of a control given as one number or as float32 [B]."""
    if v is None:
        return None, default
    if isinstance(v, torch.Tensor):
        if v.dtype != torch.float32 or v.shape != (B,) or v.get_device() != device or not v.is_contiguous():
            raise ValueError(f"{name} must be a number or a contiguous float32 [{B}] on cuda:{device}")
        return v.data_ptr(), default
    v = float(v)
    if not low <= v <= _MOST or (low == 0 and 0 < v < _LEAST):  # (1e-50 is no temperature of 0)
        raise ValueError(f"{name} = {v} is out of range")
    return None, v


def _lengths(name, t, dtype, B, device):
    if t is None:
        return None
    if t.dtype != dtype or t.shape != (B,) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{B}] on cuda:{device}")
    return t.data_ptr()


def _per_token(name, t, dtype, B, n, device):
    """(pointer, row stride) of a [n] or [B, n] operand."""
    if t is None:
        return None, 0
    shape, strides = t.shape, t.stride()
    if t.dtype != dtype or t.get_device() != device or shape != (B, n) and shape != (n,):
        raise ValueError(f"{name} must be {dtype} [{n}] or [{B}, {n}] on cuda:{device}")
    if n > 1 and strides[-1] != 1:
        raise ValueError(f"the rows of {name} must be dense")
    return t.data_ptr(), strides[0] if len(shape) == 2 else 0


_logits_ws = {}  # workspace bytes by (device, B, V, L): sizes only, no memory


def _control(logits, history, history_len, prompt_len, repetition, frequency, presence, bias, mask,
             temperature, out, tokens, seed, step):
    dtype, dev = _ck.DTYPES.get(logits.dtype), logits.get_device()
    if dtype is None or dev < 0 or logits.dim() != 2:
        raise ValueError("logits must be a CUDA tensor [B, V] of float32, bfloat16 or float16")
    _refuse_derivatives("a logit control", logits=logits, repetition=repetition, frequency=frequency,
                        presence=presence, bias=bias, temperature=temperature, out=out)
    B, V = logits.shape
    text = text_len = prompt = None
    bits = L = text_stride = 0
    if history is not None:
        it = history.dtype
        if (it is not torch.int64 and it is not torch.int32 or history.dim() != 2
                or history.shape[0] != B or history.get_device() != dev):
            raise ValueError(f"history must be int64 or int32 [{B}, L] on cuda:{dev}")
        text, bits, L = history.data_ptr(), 64 if it is torch.int64 else 32, history.shape[1]
        text_stride = _ck._rows(history, "history")
        text_len = _lengths("history_len", history_len, it, B, dev)
        prompt = _lengths("prompt_len", prompt_len, it, B, dev)
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len need a history")
    rep, rep_all = _per_row("repetition", repetition, 1.0, 1e-30, B, dev)
    freq, freq_all = _per_row("frequency", frequency, 0.0, -1e30, B, dev)
    pres, pres_all = _per_row("presence", presence, 0.0, -1e30, B, dev)
    temp, temp_all = _per_row("temperature", temperature, 1.0, 0.0, B, dev)
    bias_at, bias_stride = _per_token("bias", bias, torch.float32, B, V, dev)
    mask_at, mask_stride = _per_token("mask", mask, torch.int32, B, -(-V // 32), dev)
    out_at, out_stride = None, 0
    if out is not None:
        if out.dtype != logits.dtype or out.shape != logits.shape or out.get_device() != dev:
            raise ValueError("out must be like logits")
        out_at, out_stride = out.data_ptr(), _ck._rows(out, "out")
        _written(out)
    at = step_dev = None
    if seed is not None:
        at, step_dev = _ck._step_args(step, dev)
    ws = need = None
    if tokens is not None and V > 1024:
        key = (dev, B, V, L)
        need = _logits_ws.get(key)
        if need is None:
            if len(_logits_ws) > 4096:
                _logits_ws.clear()
            with torch.cuda.device(dev):
                need = _logits_ws[key] = _ck.ck_logits_workspace_size(B, V, L)
        if need:
            ws = torch.empty(need // 8, dtype=torch.int64, device=logits.device)
    call = _ck.LogitCall(
        logits.data_ptr(), dtype, B, V, _ck._rows(logits, "logits"), text, text_len, prompt, bits, L,
        text_stride, rep, freq, pres, temp, rep_all, freq_all, pres_all, temp_all, bias_at,
        bias_stride, mask_at, mask_stride, out_at, out_stride,
        None if tokens is None else tokens.data_ptr(), 0 if seed is None else 1,
        0 if seed is None else int(seed) & _ck._U64, at or 0, step_dev,
        None if ws is None else ws.data_ptr(), need or 0)
    if dev == _ck._get_device():
        _ck.ck_control_logits(call)
    else:
        with torch.cuda.device(dev):
            _ck.ck_control_logits(call)


def control_logits(logits, history=None, history_len=None, prompt_len=None, repetition=None,
                   frequency=None, presence=None, bias=None, mask=None, temperature=None, out=None):
    """logits [B, V] with the controls of an answering loop, in this order: the
    repetition penalty on every token of history[b, :history_len[b]] (z / r where
    z > 0, else z * r), frequency and presence penalties by its count in
    history[b, prompt_len[b]:history_len[b]], bias (float32 [V] or [B, V]), mask
    (int32 words [ceil(V / 32)] or [B, ceil(V / 32)], bit v % 32 of word v // 32
    allows token v, else -inf), then division by temperature (not where it is 0; of 16-bit
    logits a product with its reciprocal, one rounding of 32 bits more).
    Penalties and temperature are numbers or float32 [B]; history int64 or int32
    [B, L], ids outside [0, V) ignored; lengths [B] in its type."""
    got = (_ck._native or _ck.native()).control(
        logits, history, history_len, prompt_len, repetition, frequency, presence, bias, mask,
        temperature, True if out is None else out, 0, None, 0)
    if got is not None:
        return got
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    _control(logits, history, history_len, prompt_len, repetition, frequency, presence, bias, mask,
             temperature, out, None, None, 0)
    return out


def pick_tokens(logits, history=None, history_len=None, prompt_len=None, repetition=None,
                frequency=None, presence=None, bias=None, mask=None, temperature=None, seed=None,
                step=0, return_logits: bool = False, out=None):
    """The next token of each row (int64 [B]) after control_logits's controls, in
    one pass: the largest logit (the lowest token among equal ones) or, given a
    seed, a draw from their softmax in the rows whose temperature is above 0.  A
    row with no token left gives -1.  `step` as in dropout: another one for
    every token drawn.  With return_logits=True, or an `out` to write them to,
    (tokens, controlled logits)."""
    logits_too = return_logits or out is not None
    got = (_ck._native or _ck.native()).control(
        logits, history, history_len, prompt_len, repetition, frequency, presence, bias, mask,
        temperature, True if out is None and return_logits else out, 2 if logits_too else 1, seed, step)
    if got is not None:
        return got
    if out is None and return_logits:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    tokens = torch.empty(logits.shape[:1], dtype=torch.int64, device=logits.device)
    _control(logits, history, history_len, prompt_len, repetition, frequency, presence, bias, mask,
             temperature, out, tokens, seed, step)
    return tokens if out is None else (tokens, out)
