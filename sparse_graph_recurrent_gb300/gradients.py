"""The global norm of a model's gradients, and their clipping, between a backward pass and
an update (ck_sgd_update, ck_adam_update or an optimizer of torch's).

    norm = clip_gradients([p.grad for p in params], 1.0)

Every call enqueues its kernels on the current stream and returns without waiting: the norm
stays on the device, and the call can be captured.
"""
from __future__ import annotations

import torch

from . import _ck
from .readout import _refuse_derivatives, _written

__all__ = ["grad_norm", "clip_gradients"]


def _tensors(grads, name):
    if isinstance(grads, torch.Tensor):
        grads = [grads]
    some = list(grads)
    for t in some:
        if t is None:
            continue
        if not t.is_cuda or t.dtype not in _ck.DTYPES or t.layout != torch.strided:
            raise ValueError(f"{name} are CUDA tensors of float32, bfloat16 or float16")
    return some


def _dense(t):
    """Whether t's elements fill a stretch of memory, in whatever order."""
    if t.is_contiguous():
        return True
    at = 1
    for s, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n != 1):
        if s != at:
            return False
        at *= n
    return True


def _direct(g, o):
    """Whether the C entry can take g and its output o as they are."""
    return _dense(g) and (o is g or o.stride() == g.stride() and o.is_neg() == g.is_neg())


class _Span:
    """The bytes from a tensor's first to its last, [lo, hi)."""

    def __init__(self, t, written):
        self.size, self.written = t.element_size(), written
        self.axes = [(s * self.size, n) for n, s in zip(t.shape, t.stride()) if n != 1]
        self.lo = t.data_ptr()
        self.hi = self.lo + sum(s * (n - 1) for s, n in self.axes) + self.size

    def of_every(self, m):
        """The bytes that it takes of every m, from where it begins on, or more than m."""
        return self.size + sum(s * (n - 1) if s < m else m for s, n in self.axes if s % m)

    def beside(self, other):
        """Whether another, that begins no earlier, takes others of every so many bytes: columns of
        one array, or its rows by turns."""
        for m in {s for s, _ in self.axes + other.axes if s}:
            apart = (other.lo - self.lo) % m
            if self.of_every(m) <= apart and apart + other.of_every(m) <= m:
                return True
        return False


def _refuse_shared(pairs):
    """Refuses tensors that share memory where one of them is written, or may.  (Of dense ones the
    C entry looks after that; others go there by way of copies.)"""
    spans = []
    for g, o in pairs:
        if not g.numel():
            continue
        read, written = _Span(g, False), _Span(o, True)
        if any(not s for s, _ in written.axes):
            raise ValueError("elements of a tensor that is written share memory")
        spans.append(written)
        if (read.lo, read.axes) != (written.lo, written.axes):  # (not in its own place)
            spans.append(read)
    spans.sort(key=lambda s: s.lo)
    for i, a in enumerate(spans):
        for b in spans[i + 1:]:
            if b.lo >= a.hi:
                break
            if (a.written or b.written) and not a.beside(b):
                raise ValueError("two tensors share memory that is written")


def _space(array, device):
    return torch.empty(_ck.ck_clip_workspace_size(array) // 8, dtype=torch.int64, device=device)


def _one_device(some):
    device = some[0].get_device()
    if any(t.get_device() != device for t in some):
        raise ValueError("gradients must be on one device")
    return some[0].device


def grad_norm(grads):
    """The root of the sum of the squares of all elements of a tensor or of several
    (float32, bfloat16 or float16, mixed as they are; None is skipped): a float32 scalar
    on the device, off by 2e-6 of it at most.  No tensor at all gives 0 on the current device."""
    norm = (_ck._native or _ck.native()).clip(grads, None, None)
    if norm is not None:
        return norm
    some = [t for t in _tensors(grads, "gradients") if t is not None]
    for t in some:
        _refuse_derivatives("grad_norm", gradient=t)
    norm = torch.empty((), dtype=torch.float32, device=some[0].device if some else "cuda")
    device = _one_device(some) if some else norm.device
    flat = [t.detach() if _dense(t) else t.detach().contiguous() for t in some]
    with torch.cuda.device(device):
        array = _ck.gradient_list(flat)
        _ck.ck_grad_norm(array, norm, _space(array, device))
    return norm


def clip_gradients(grads, max_norm: float, out=None):
    """grad_norm of the tensors, which are then multiplied in place by
    min(1, max_norm / (norm + 1e-6)): by nothing where the norm is small enough.  `out`, a
    tensor or as many as there are gradients, of their types and shapes, receives the
    products instead.  None is skipped.  Tensors that share memory are refused where it
    is written, and so are strided ones of which that cannot be told from their strides."""
    norm = (_ck._native or _ck.native()).clip(grads, max_norm, out) if max_norm is not None else None
    if norm is not None:
        return norm
    single = isinstance(grads, torch.Tensor)
    some = _tensors(grads, "gradients")
    to = some if out is None else _tensors(out, "out")
    if len(to) != len(some) or single != isinstance(out, torch.Tensor) and out is not None:
        raise ValueError("out holds as many tensors as there are gradients")
    pairs = [(g, o) for g, o in zip(some, to) if g is not None]
    for g, o in pairs:
        _refuse_derivatives("clip_gradients", gradient=g, out=o)
        if o is None or o.dtype != g.dtype or o.shape != g.shape or o.device != g.device:
            raise ValueError("out is like the gradients")
    device = _one_device([g for g, _ in pairs]) if pairs else torch.device("cuda", torch.cuda.current_device())
    norm = torch.empty((), dtype=torch.float32, device=device)
    ins, outs, back = [], [], []
    if not all(_direct(g, o) for g, o in pairs):
        _refuse_shared(pairs)
    for g, o in pairs:
        g, own = g.detach(), o is g
        if not _direct(g, o):
            # by way of a dense one: a copy of the gradient, or where the gradient is itself
            # dense in order, other memory beside it
            aim, copied, g = o, not g.is_contiguous() or g.is_neg(), g.resolve_neg().contiguous()
            if not o.is_contiguous() or own or o.is_neg():
                o, own = g if copied else torch.empty_like(g), False
                back.append((aim, o))
        ins.append(g)
        outs.append(g if own else o.detach())
    with torch.cuda.device(device):
        array = _ck.gradient_list(ins, outs)
        _ck.ck_clip_gradients(array, max_norm, norm, _space(array, device))
        for o, g in back:
            o.detach().copy_(g)
    for _, o in pairs:
        _written(o)
    return norm
