"""A linear recurrence whose leak, or decay, is given for every step: the layer that a
recurrent token model puts beside or on top of sparse_recurrence, in its layout [T, B, N].

    out, state = gated_recurrence(x, gate, state0)                 # training, differentiable
    out, state = gated_recurrence(x[None], gate[None], state)      # answering, one step

Every call enqueues its kernels on the current stream and returns without waiting.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _ck
from .readout import _followed

__all__ = ["gated_recurrence", "gated_recurrence_forward", "gated_recurrence_backward"]


def _steps(t, name, shape, dtype, device):
    """(t with dense nodes, its strides of steps and sequences)."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on cuda:{device}, not {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    t = t.resolve_neg()
    if t.shape[2] > 1 and t.stride(2) != 1:
        t = t.contiguous()
    return t, t.stride(0), t.stride(1)


def _state(t, name, B, N, device):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (B, N) or t.get_device() != device:
        raise ValueError(f"{name} must be float32 [{B}, {N}] on cuda:{device}, not {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    return t.resolve_neg().contiguous()


def _call(x, gate, lengths, form):
    """The arguments that both directions take, and what has to live until they are enqueued."""
    if x.dtype not in _ck.DTYPES or not x.is_cuda or x.dim() != 3:
        raise ValueError("x must be a CUDA tensor [T, B, N] of float32, bfloat16 or float16")
    if form not in _ck.GATED_FORMS:
        raise ValueError(f"form is 'leak' or 'decay', not {form!r}")
    device, (T, B, N) = x.get_device(), x.shape
    x, xt, xb = _steps(x, "x", x.shape, x.dtype, device)
    gate, gt, gb = _steps(gate, "gate", x.shape, x.dtype, device)
    if lengths is not None:
        if lengths.dtype != torch.int64 or lengths.shape != (B,) or lengths.get_device() != device:
            raise ValueError(f"lengths must be int64 [{B}] on cuda:{device}")
        lengths = lengths.contiguous()
    call = _ck.GatedCall(x=x.data_ptr(), gate=gate.data_ptr(), dtype=_ck.DTYPES[x.dtype], form=_ck.GATED_FORMS[form],
                         T=T, B=B, N=N, x_step=xt, x_row=xb, gate_step=gt, gate_row=gb,
                         lengths=None if lengths is None else lengths.data_ptr())
    return call, (x, gate, lengths), device, (T, B, N)


_sizes = {}  # (bytes of kept, of workspace) by (device, T, B, N): sizes only, no memory


def _space(device, T, B, N):
    key = (device, T, B, N)
    got = _sizes.get(key)
    if got is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        with torch.cuda.device(device):
            got = _sizes[key] = _ck.ck_gated_sizes(T, B, N)
    return got


def _workspace(call, need, like):
    ws = None
    if need:
        ws = torch.empty(need // 8, dtype=torch.int64, device=like.device)
        call.workspace, call.workspace_bytes = ws.data_ptr(), need
    return ws


def _enqueue(entry, call, device):
    if device == _ck._get_device():
        entry(call)
    else:
        with torch.cuda.device(device):
            entry(call)


def _forward(x, gate, state0, lengths, form, keep):
    call, held, device, (T, B, N) = _call(x, gate, lengths, form)
    state0 = _state(state0, "state0", B, N, device)
    out = torch.empty((T, B, N), dtype=x.dtype, device=x.device)
    state = torch.empty((B, N), dtype=torch.float32, device=x.device)
    kept_bytes, need = _space(device, T, B, N)
    kept = torch.empty(kept_bytes // 4, dtype=torch.float32, device=x.device) if keep else None
    ws = _workspace(call, need, x)
    call.state0 = None if state0 is None else state0.data_ptr()
    call.out, call.state = out.data_ptr(), state.data_ptr()
    if keep:
        call.kept = kept.data_ptr()
    _enqueue(_ck.ck_gated_forward, call, device)
    del held, ws
    return out, state, kept


def gated_recurrence_forward(x, gate, state0=None, lengths=None, form: str = "leak"):
    """gated_recurrence without autograd: (out, state, kept), kept for
    gated_recurrence_backward (32-bit states at every 8th step)."""
    got = (_ck._native or _ck.native()).gated(x, gate, state0, lengths, form, True)
    if got is not None:
        return got
    x, gate = x.detach(), gate.detach()
    return _forward(x, gate, None if state0 is None else state0.detach(), lengths, form, True)


def _backward(x, gate, kept, d_out, d_state, lengths, form, want=(True, True, True)):
    got = (_ck._native or _ck.native()).gated_backward(x, gate, kept, d_out, d_state, lengths, form, *want)
    if got is not None:
        return got
    call, held, device, (T, B, N) = _call(x, gate, lengths, form)
    kept_bytes, need = _space(device, T, B, N)
    if kept.dtype != torch.float32 or kept.numel() * 4 != kept_bytes or kept.get_device() != device or not kept.is_contiguous():
        raise ValueError("kept is not what gated_recurrence_forward returned for these sizes")
    if d_out is not None:
        d_out, call.d_out_step, call.d_out_row = _steps(d_out, "d_out", x.shape, x.dtype, device)
        call.d_out = d_out.data_ptr()
    d_state = _state(d_state, "d_state", B, N, device)
    call.d_state = None if d_state is None else d_state.data_ptr()
    call.kept = kept.data_ptr()
    dx = torch.empty((T, B, N), dtype=x.dtype, device=x.device) if want[0] else None
    dgate = torch.empty((T, B, N), dtype=x.dtype, device=x.device) if want[1] else None
    dstate0 = torch.empty((B, N), dtype=torch.float32, device=x.device) if want[2] else None
    call.dx, call.dgate, call.d_state0 = (None if t is None else t.data_ptr() for t in (dx, dgate, dstate0))
    ws = _workspace(call, need, x)
    _enqueue(_ck.ck_gated_backward, call, device)
    del held, ws
    return dx, dgate, dstate0


def gated_recurrence_backward(x, gate, kept, d_out, d_state=None, lengths=None, form: str = "leak"):
    """(dx, dgate, dstate0) from the gradients of gated_recurrence_forward's out and state
    (either may be None: zeros), for the same x, gate, lengths and form."""
    got = (_ck._native or _ck.native()).gated_backward(x, gate, kept, d_out, d_state, lengths, form, True, True, True)
    if got is not None:
        return got
    return _backward(x.detach(), gate.detach(), kept, None if d_out is None else d_out.detach(),
                     None if d_state is None else d_state.detach(), lengths, form)


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, state0, lengths, form):
        ctx.set_materialize_grads(False)
        out, state, kept = gated_recurrence_forward(x, gate, state0, lengths, form)
        ctx.save_for_backward(x, gate, kept, lengths)
        ctx.form = form
        return out, state

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_state):
        if d_out is None and d_state is None:
            return None, None, None, None, None
        x, gate, kept, lengths = ctx.saved_tensors
        got = _backward(x.detach(), gate.detach(), kept, d_out, d_state, lengths, ctx.form, ctx.needs_input_grad[:3])
        return (*got, None, None)


def gated_recurrence(x, gate, state0=None, lengths=None, form: str = "leak"):
    """(out [T, B, N], state [B, N]): the states h_t after every step and the last one.
    form "leak": h_t = (1 - l) h_{t-1} + l x_t with l = sigmoid(gate_t), the blend of
    sparse_recurrence with a leak for every step; "decay": h_t = gate_t h_{t-1} + x_t.
    x is float32, bfloat16 or float16, gate is of its type and of its shape or expands to
    it; state0 is float32 [B, N] (zeros by default) and so is state, whatever x's type.
    lengths, int64 [B]: from step lengths[b] on the state stays as it is, out is 0 and x
    and gate do not matter.  Decays may lie beyond 1 as long as the states stay inside 32 bits;
    where long sequences are cut along their steps, runs whose product of decays does not are
    gone through step by step, which is slow.  Differentiable (once) in x, gate and state0."""
    got = (_ck._native or _ck.native()).gated(x, gate, state0, lengths, form, False)
    if got is not None:
        return got[:2]
    if gate.shape != x.shape:
        gate = gate.expand(x.shape)
    if _followed(x) or _followed(gate) or state0 is not None and _followed(state0):
        return _GatedRecurrence.apply(x, gate, state0, lengths, form)
    return _forward(x, gate, state0, lengths, form, False)[:2]
