"""ctypes binding of libck's C ABI (include/ck.h): argument marshalling only.

Every function here has the name of the C entry point it calls and takes torch
CUDA tensors in place of raw device pointers.  All computation happens in the
library's CUDA kernels; if the library cannot be built or loaded this module
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from contextlib import nullcontext

import torch

from . import build as _build

CK_OK = 0
STATUS = {0: "CK_OK", 1: "CK_ERR_INVALID_ARG", 2: "CK_ERR_CUDA", 3: "CK_ERR_OUT_OF_MEMORY",
          4: "CK_ERR_TIMEOUT", 5: "CK_ERR_WORKSPACE", 6: "CK_ERR_INTERNAL",
          7: "CK_ERR_UNSUPPORTED"}
(OPT_PERSISTENT, OPT_BARRIER_TIMEOUT_NS, OPT_TEST_BARRIER_EXTRA, OPT_GRAPH_IN_SMEM,
 OPT_RECOMPUTE_STEPS, OPT_ROWS_IN_SMEM, OPT_TEST_BOUNDS_PROBE, OPT_TILED) = range(8)
GRAPH_EDGES_IN_HOST_MEMORY, GRAPH_TILING = 1, 2  # ck_graph_flag
# ck_barrier_scheme (ck_probe_grid_barrier)
(BARRIER_COUNTER, BARRIER_COUNTER_RETURNING, BARRIER_COUNTER_RELAXED, BARRIER_FLAG,
 BARRIER_FLAGS8, BARRIER_CLUSTER_SYNC, BARRIER_CLUSTER_MBARRIER) = range(7)
PROBE_BARRIER_WORDS = 16384
PHASE_PROFILE_CTAS, PHASE_PROFILE_WORDS = 1024, 8  # ck_phase_profile_read
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # ck_dtype
INT4_GROUPS = (32, 64, 128)
GATED_FORMS = {"leak": 0, "decay": 1}  # ck_gated_form

_lib = None


class LogitCall(ctypes.Structure):
    """ck_logit_call: the arguments of ck_control_logits."""
    _p, _i, _f, _u = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64
    _fields_ = [("logits", _p), ("dtype", _i), ("B", _i), ("V", _i), ("logits_stride", _i),
                ("history", _p), ("history_len", _p), ("prompt_len", _p),
                ("history_bits", _i), ("L", _i), ("history_stride", _i),
                ("repetition", _p), ("frequency", _p), ("presence", _p), ("temperature", _p),
                ("repetition_all", _f), ("frequency_all", _f), ("presence_all", _f),
                ("temperature_all", _f),
                ("bias", _p), ("bias_stride", _i), ("mask", _p), ("mask_stride", _i),
                ("out", _p), ("out_stride", _i), ("tokens", _p), ("sample", _i),
                ("seed", _u), ("step", _u), ("step_dev", _p), ("workspace", _p),
                ("workspace_bytes", _i)]


class GatedCall(ctypes.Structure):
    """ck_gated_call: the arguments of ck_gated_forward and ck_gated_backward."""
    _p, _i = ctypes.c_void_p, ctypes.c_int64
    _fields_ = [("x", _p), ("gate", _p), ("dtype", _i), ("form", _i), ("T", _i), ("B", _i), ("N", _i),
                ("x_step", _i), ("x_row", _i), ("gate_step", _i), ("gate_row", _i), ("state0", _p),
                ("lengths", _p), ("out", _p), ("state", _p), ("kept", _p), ("d_out", _p),
                ("d_out_step", _i), ("d_out_row", _i), ("d_state", _p), ("dx", _p), ("dgate", _p),
                ("d_state0", _p), ("workspace", _p), ("workspace_bytes", _i)]


class Gradient(ctypes.Structure):
    """ck_gradient: a tensor of ck_grad_norm and ck_clip_gradients."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int64)]


class BeamCall(ctypes.Structure):
    """ck_beam_call: the arguments of ck_beam_select."""
    _p, _i = ctypes.c_void_p, ctypes.c_int64
    _fields_ = [("logits", _p), ("dtype", _i), ("B", _i), ("K", _i), ("V", _i), ("logits_row", _i),
                ("logits_beam", _i), ("scores", _p), ("ended", _p), ("end_token", _i), ("beams", _i),
                ("scores_out", _p), ("parents", _p), ("tokens", _p), ("ended_out", _p), ("workspace", _p),
                ("workspace_bytes", _i)]


class BeamState(ctypes.Structure):
    """ck_beam_state: an array of ck_reorder_states."""
    _p, _i = ctypes.c_void_p, ctypes.c_int64
    _fields_ = [("in_", _p), ("out", _p), ("bytes", _i), ("in_row", _i), ("in_beam", _i), ("out_row", _i),
                ("out_beam", _i)]


class CKError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS.get(status, str(status))


def library_variant():
    """The library variant this process loads: None (libck.so), "bounds"
    (libck_bounds.so, the bounds-checked build) or "prof" (libck_prof.so, with
    the phase profile), from CK_LIBRARY_VARIANT."""
    return os.environ.get("CK_LIBRARY_VARIANT") or None


def library_path() -> str:
    return _build.lib_path(library_variant())


def load() -> ctypes.CDLL:
    """Load the library, building it with nvcc first if it is missing or stale."""
    global _lib, _native
    if _lib is not None:
        return _lib
    path = _build.build(variant=library_variant())
    if not os.path.exists(path):
        raise ImportError(f"libck.so not found at {path}")
    lib = ctypes.CDLL(path)
    p, i64, sz, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint64
    psz = ctypes.POINTER(ctypes.c_size_t)
    pi64 = ctypes.POINTER(ctypes.c_int64)
    sig = {
        "ck_graph_create": [p, p, i64, i64, p, i64, p, ctypes.POINTER(p)],
        "ck_graph_create_flags": [p, p, i64, i64, p, i64, ctypes.c_uint32, p, ctypes.POINTER(p)],
        "ck_graph_destroy": [p],
        "ck_graph_info": [p, pi64, pi64, pi64],
        "ck_graph_memory": [p, psz, psz],
        "ck_graph_tiling": [p, ctypes.c_int, pi64],
        "ck_graph_export_tiling": [p, ctypes.c_int, p, p, p, p, p, p],
        "ck_graph_export": [p, p, p, p, p, p, p, p, p],
        "ck_workspace_size": [p, i64, i64, i64, psz, psz],
        "ck_forward": [p, p, p, p, p, p, i64, i64, i64, p, p, sz, p, sz, p],
        "ck_backward": [p, p, p, i64, i64, i64, p, sz, p, p, p, p, p, p, p, sz, p],
        "ck_workspace_size_recompute": [p, i64, i64, i64, psz, psz],
        "ck_sgd_update": [p, p, i64, ctypes.c_float, p],
        "ck_adam_update": [p, p, p, p, i64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                           ctypes.c_float, p, p],
        "ck_step_advance": [p, p],
        "ck_forward_checkpointed": [p, p, p, p, p, p, i64, i64, i64, p, p, sz, p, sz, p],
        "ck_backward_recompute": [p, p, p, p, p, i64, i64, i64, p, sz, p, p, p, p, p, p, p, sz, p],
        "ck_query_status": [p, p],
        "ck_query_status_static": [p],
        "ck_set_option": [ctypes.c_int, i64],
        "ck_dropout": [p, p, i64, *[i64] * 9, i64, ctypes.c_double, u64, u64, p, p],
        "ck_int4_matvec": [p, i64, i64, i64, i64, p, i64, i64, p, i64, i64, p, i64, p, i64, p, i64,
                           p, sz, p],
        "ck_int4_workspace_size": [i64, i64, i64, i64, i64, psz],
        "ck_int4_quantize": [p, i64, i64, i64, i64, i64, i64, p, i64, p, i64, i64, p, i64, p],
        "ck_control_logits": [ctypes.POINTER(LogitCall), p],
        "ck_logits_workspace_size": [i64, i64, i64, psz],
        "ck_gated_sizes": [i64, i64, i64, psz, psz],
        "ck_gated_forward": [ctypes.POINTER(GatedCall), p],
        "ck_gated_backward": [ctypes.POINTER(GatedCall), p],
        "ck_clip_workspace_size": [ctypes.POINTER(Gradient), i64, psz],
        "ck_grad_norm": [ctypes.POINTER(Gradient), i64, p, p, i64, p],
        "ck_clip_gradients": [ctypes.POINTER(Gradient), i64, ctypes.c_double, p, p, i64, p],
        "ck_beam_workspace_size": [i64, i64, i64, i64, i64, psz],
        "ck_beam_select": [ctypes.POINTER(BeamCall), p],
        "ck_reorder_states": [ctypes.POINTER(BeamState), i64, p, i64, i64, i64, p],
        "ck_forward_static_scratch": [p, p, p, p, p, p, i64, i64, i64, p, p, sz, p],
        "ck_probe_read": [p, sz, i64, p, p],
        "ck_probe_gather": [p, i64, i64, p, i64, p, p],
        "ck_probe_read_shape": [p, sz, i64, i64, i64, i64, i64, p, p],
        "ck_probe_grid_barrier": [i64, i64, i64, i64, i64, p, p, p, p],
        "ck_phase_profile_read": [p, i64, i64],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.ck_get_option.argtypes = [ctypes.c_int]
    lib.ck_get_option.restype = i64
    lib.ck_last_launch_count.argtypes = []
    lib.ck_last_launch_count.restype = i64
    lib.ck_status_string.argtypes = [ctypes.c_int]
    lib.ck_status_string.restype = ctypes.c_char_p
    lib.ck_last_error_message.argtypes = []
    lib.ck_last_error_message.restype = ctypes.c_char_p
    native = _load_native(lib)
    _lib, _native = lib, native
    return lib


_native = None


class _PythonForms:
    """In the place of ck_binding where that cannot be had: leaves every call to its Python form."""

    @staticmethod
    def dropout(*args):
        return None

    int4_matvec = control = gated = gated_backward = clip = beam = reorder = dropout


def _load_native(lib):
    """The module ck_binding (the token model's operators' short way from Python), built first if
    it is missing or stale, with this library's entries.  All else works without it."""
    import importlib.machinery
    import importlib.util
    try:
        loader = importlib.machinery.ExtensionFileLoader("ck_binding", _build.build_binding())
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("ck_binding", loader))
        loader.exec_module(module)
    except (ImportError, OSError, RuntimeError) as e:  # no compiler, no headers, another interpreter's
        warnings.warn("the token model's operators are called through ctypes, some microseconds "
                      f"slower, as ck_binding cannot be had: {e}", RuntimeWarning, stacklevel=3)
        return _PythonForms
    entry = lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value  # noqa: E731
    module.bind(tuple(entry("ck_" + name) for name in (
        "dropout", "int4_matvec", "int4_workspace_size", "control_logits", "logits_workspace_size", "gated_sizes",
        "gated_forward", "gated_backward", "clip_workspace_size", "grad_norm", "clip_gradients",
        "beam_workspace_size", "beam_select", "reorder_states")), _check)
    return module


def native():
    """The module ck_binding, or what stands in its place."""
    if _native is None:
        load()
    return _native


def _check(status: int):
    if status != CK_OK:
        raise CKError(status, load().ck_last_error_message().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_U64 = (1 << 64) - 1


# The current device and its current stream as plain integers.  The calls torch's own
# code generators use cost 0.1 us each, the public ones 0.3 and 3, on a path of about
# 7; the public ways stay for a torch that lacks the others.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(stream):
    return _get_raw_stream(_get_device()) if stream is None else stream.cuda_stream


def _need(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _shapes(handle, B: int, T: int, **tensors):
    """The library sees only pointers, so every tensor's shape is checked here
    against the graph's N, E, n_in and the call's B, T."""
    N, E, n_in = ck_graph_info(handle)
    want = {"edge_values": (E,), "d_edge_values": (E,), "leak": (N,), "d_leak": (N,),
            "bias": (N,), "d_bias": (N,), "drives": (T, n_in, B), "d_drives": (T, n_in, B),
            "state0": (B, N), "d_state0": (B, N), "states_out": (T, B, N), "d_states": (T, B, N)}
    for name, t in tensors.items():
        if t is None:
            if name in ("drives", "d_drives") and n_in == 0:
                continue
            raise ValueError(f"{name} is required")
        if tuple(t.shape) != want[name]:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want[name]}")


def ck_graph_create(src, dst, num_nodes: int, input_nodes, stream=None, flags: int = 0):
    """ck_graph_create, or ck_graph_create_flags when flags is non-zero."""
    for t, n in ((src, "src"), (dst, "dst"), (input_nodes, "input_nodes")):
        _need(t, torch.int64, n)
    h = ctypes.c_void_p()
    n_in = 0 if input_nodes is None else input_nodes.numel()
    args = (_ptr(src), _ptr(dst), src.numel(), num_nodes, _ptr(input_nodes) if n_in else None, n_in)
    if flags:
        _check(load().ck_graph_create_flags(*args, int(flags), _stream(stream), ctypes.byref(h)))
    else:
        _check(load().ck_graph_create(*args, _stream(stream), ctypes.byref(h)))
    return h


def ck_graph_destroy(handle):
    _check(load().ck_graph_destroy(handle))


def ck_graph_info(handle):
    n, e, k = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(load().ck_graph_info(handle, ctypes.byref(n), ctypes.byref(e), ctypes.byref(k)))
    return n.value, e.value, k.value


def ck_graph_export(handle, device=None, stream=None):
    N, E, _ = ck_graph_info(handle)
    dev = device or torch.device("cuda", torch.cuda.current_device())
    mk = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    out = dict(row_ptr=mk(N + 1), col=mk(E), perm=mk(E), rowT_ptr=mk(N + 1), colT=mk(E),
               permT=mk(E), slot=mk(N))
    _check(load().ck_graph_export(handle, *(_ptr(out[k]) for k in
                                            ("row_ptr", "col", "perm", "rowT_ptr", "colT",
                                             "permT", "slot")), _stream(stream)))
    return out


def ck_workspace_size(handle, B: int, T: int, microsteps: int):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().ck_workspace_size(handle, B, T, microsteps, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def ck_forward(handle, edge_values, leak, bias, drives, state0, microsteps, states_out,
               saved, scratch, stream=None):
    for t, n in ((edge_values, "edge_values"), (leak, "leak"), (bias, "bias"),
                 (drives, "drives"), (state0, "state0"), (states_out, "states_out")):
        _need(t, torch.float32, n)
    B = state0.shape[0]
    T = states_out.shape[0]
    _shapes(handle, B, T, edge_values=edge_values, leak=leak, bias=bias, drives=drives,
            state0=state0, states_out=states_out)
    _check(load().ck_forward(handle, _ptr(edge_values), _ptr(leak), _ptr(bias),
                             _ptr(drives) if drives is not None and drives.numel() else None,
                             _ptr(state0), B, T, microsteps, _ptr(states_out),
                             _ptr(saved), saved.numel() * saved.element_size(),
                             _ptr(scratch), scratch.numel() * scratch.element_size(),
                             _stream(stream)))


def ck_backward(handle, edge_values, leak, B, T, microsteps, saved, d_states, d_edge_values,
                d_leak, d_bias, d_drives, d_state0, scratch, stream=None):
    for t, n in ((edge_values, "edge_values"), (leak, "leak"), (d_states, "d_states"),
                 (d_edge_values, "d_edge_values"), (d_leak, "d_leak"), (d_bias, "d_bias"),
                 (d_drives, "d_drives"), (d_state0, "d_state0")):
        _need(t, torch.float32, n)
    _shapes(handle, B, T, edge_values=edge_values, leak=leak, d_states=d_states,
            d_edge_values=d_edge_values, d_leak=d_leak, d_bias=d_bias, d_drives=d_drives,
            d_state0=d_state0)
    _check(load().ck_backward(handle, _ptr(edge_values), _ptr(leak), B, T, microsteps,
                              _ptr(saved), saved.numel() * saved.element_size(),
                              _ptr(d_states), _ptr(d_edge_values), _ptr(d_leak), _ptr(d_bias),
                              _ptr(d_drives) if d_drives is not None and d_drives.numel() else None,
                              _ptr(d_state0), _ptr(scratch),
                              scratch.numel() * scratch.element_size(), _stream(stream)))


def ck_sgd_update(param, grad, lr: float, stream=None):
    _need(param, torch.float32, "param")
    _need(grad, torch.float32, "grad")
    if param.shape != grad.shape:
        raise ValueError("param and grad differ in shape")
    _check(load().ck_sgd_update(_ptr(param), _ptr(grad), param.numel(), float(lr),
                                _stream(stream)))


def ck_adam_update(param, grad, m, v, step, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, stream=None):
    """Adam at the step number held by the device int64 tensor `step`."""
    for t, name in ((param, "param"), (grad, "grad"), (m, "m"), (v, "v")):
        _need(t, torch.float32, name)
        if t.shape != param.shape:
            raise ValueError(f"{name} differs in shape from param")
    _need(step, torch.int64, "step")
    _check(load().ck_adam_update(_ptr(param), _ptr(grad), _ptr(m), _ptr(v), param.numel(),
                                 float(lr), float(beta1), float(beta2), float(eps), _ptr(step),
                                 _stream(stream)))


def ck_step_advance(step, stream=None):
    _need(step, torch.int64, "step")
    _check(load().ck_step_advance(_ptr(step), _stream(stream)))


def ck_workspace_size_recompute(handle, B: int, T: int, microsteps: int):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().ck_workspace_size_recompute(handle, B, T, microsteps, ctypes.byref(a),
                                              ctypes.byref(b)))
    return a.value, b.value


def ck_forward_checkpointed(handle, edge_values, leak, bias, drives, state0, microsteps,
                            states_out, ckpt, scratch, stream=None):
    for t, n in ((edge_values, "edge_values"), (leak, "leak"), (bias, "bias"),
                 (drives, "drives"), (state0, "state0"), (states_out, "states_out")):
        _need(t, torch.float32, n)
    B = state0.shape[0]
    T = states_out.shape[0]
    _shapes(handle, B, T, edge_values=edge_values, leak=leak, bias=bias, drives=drives,
            state0=state0, states_out=states_out)
    _check(load().ck_forward_checkpointed(
        handle, _ptr(edge_values), _ptr(leak), _ptr(bias),
        _ptr(drives) if drives is not None and drives.numel() else None, _ptr(state0), B, T,
        microsteps, _ptr(states_out), _ptr(ckpt), ckpt.numel() * ckpt.element_size(),
        _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)))


def ck_backward_recompute(handle, edge_values, leak, bias, drives, B, T, microsteps, ckpt,
                          d_states, d_edge_values, d_leak, d_bias, d_drives, d_state0, scratch,
                          stream=None):
    for t, n in ((edge_values, "edge_values"), (leak, "leak"), (bias, "bias"),
                 (drives, "drives"), (d_states, "d_states"), (d_edge_values, "d_edge_values"),
                 (d_leak, "d_leak"), (d_bias, "d_bias"), (d_drives, "d_drives"),
                 (d_state0, "d_state0")):
        _need(t, torch.float32, n)
    _shapes(handle, B, T, edge_values=edge_values, leak=leak, bias=bias, drives=drives,
            d_states=d_states, d_edge_values=d_edge_values, d_leak=d_leak, d_bias=d_bias,
            d_drives=d_drives, d_state0=d_state0)
    has_in = drives is not None and drives.numel()
    _check(load().ck_backward_recompute(
        handle, _ptr(edge_values), _ptr(leak), _ptr(bias), _ptr(drives) if has_in else None, B, T,
        microsteps, _ptr(ckpt), ckpt.numel() * ckpt.element_size(), _ptr(d_states),
        _ptr(d_edge_values), _ptr(d_leak), _ptr(d_bias),
        _ptr(d_drives) if d_drives is not None and d_drives.numel() else None, _ptr(d_state0),
        _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)))


def _step_args(step, device: int):
    """(host step, device pointer) of a step given as an int or a device int64[1]."""
    if isinstance(step, torch.Tensor):
        if step.dtype != torch.int64 or step.numel() != 1 or step.get_device() != device:
            raise ValueError(f"a step tensor is one int64 on cuda:{device}")
        return 0, step.data_ptr()
    return int(step) & _U64, None


def ck_dropout(x, y, n0, n1, n2, x0, x1, x2, p: float, seed: int, step=0, locked=False,
               stream=None):
    """x as [n0][n1][n2] with strides x0, x1, x2 in elements; y contiguous in that order."""
    dtype, device = DTYPES.get(x.dtype), x.get_device()
    if dtype is None or device < 0 or y.dtype != x.dtype or y.get_device() != device:
        raise ValueError("dropout takes CUDA tensors of float32, bfloat16 or float16, out like x")
    dev = None
    if type(step) is not int:
        step, dev = _step_args(step, device)
    status = (_lib or load()).ck_dropout(
        x.data_ptr(), y.data_ptr(), dtype, n0, n1, n2, x0, x1, x2, n1 * n2, n2, 1, bool(locked), float(p),
        int(seed) & _U64, step & _U64, dev,
        _get_raw_stream(_get_device()) if stream is None else stream.cuda_stream)
    if status:
        _check(status)


def _like(t, device: int, dtype, shape, name):
    if t.get_device() != device or (dtype is not None and t.dtype != dtype) or t.shape != shape:
        raise ValueError(f"{name} must be {dtype or 'a tensor'} of shape {tuple(shape)} on "
                         f"cuda:{device}, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, name):
    """Elements between the rows of a 2-D tensor with dense rows."""
    (n, m), (pitch, one) = t.shape, t.stride()
    if one != 1 and m > 1:
        raise ValueError(f"the rows of {name} must be dense")
    return pitch if n > 1 else m


def ck_int4_workspace_size(dtype, M: int, K: int, V: int, group: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ck_int4_workspace_size(DTYPES[dtype], M, K, V, group, ctypes.byref(n)))
    return n.value


_int4_ws = {}  # bytes by (device, dtype, M, K, V, group): sizes only, no memory


def ck_int4_matvec(x, qweight, scales, zeros, bias, group: int, y, stream=None):
    """x [M, K], qweight uint8 [V, (K + 1) / 2], scales and zeros [V, ceil(K / group)], y [M, V].
    The workspace is taken from torch's allocator on the stream that the product runs on."""
    if x.dtype not in DTYPES or scales.dtype not in DTYPES or not x.is_cuda:
        raise ValueError("x and scales are CUDA tensors of float32, bfloat16 or float16")
    if group not in INT4_GROUPS:
        raise ValueError(f"group_size must be one of {INT4_GROUPS}, not {group}")
    if x.dim() != 2 or qweight.dim() != 2 or scales.dim() != 2:
        raise ValueError("x, qweight and scales are 2-D")
    M, K = x.shape
    V, dev = qweight.shape[0], x.get_device()
    if K < 1:
        raise ValueError("x needs at least one column")
    G = -(-K // group)
    _like(qweight, dev, torch.uint8, (V, (K + 1) // 2), "qweight")
    _like(scales, dev, None, (V, G), "scales")
    _like(y, dev, x.dtype, (M, V), "out")
    if zeros is not None:
        _like(zeros, dev, torch.uint8, (V, G), "zeros")
    if bias is not None:
        _like(bias, dev, torch.float32, (V,), "bias")
        if not bias.is_contiguous():
            raise ValueError("bias must be contiguous")
    # a single row may be of any pitch
    pitch = _rows(qweight, "qweight") if V > 1 else -(-qweight.shape[1] // 16) * 16
    if qweight.shape[1] > 1 and qweight.stride(1) != 1:
        raise ValueError("the rows of qweight must be dense")
    key = (dev, x.dtype, M, K, V, group)
    need = _int4_ws.get(key)
    if need is None:
        if len(_int4_ws) > 4096:
            _int4_ws.clear()
        need = _int4_ws[key] = ck_int4_workspace_size(x.dtype, M, K, V, group)
    ws = None
    if need:
        # of the stream that uses it: another's block may still have work of its own pending
        with nullcontext() if stream is None else torch.cuda.stream(stream):
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    status = (_lib or load()).ck_int4_matvec(
        x.data_ptr(), DTYPES[x.dtype], M, K, _rows(x, "x"), qweight.data_ptr(), V, pitch,
        scales.data_ptr(), DTYPES[scales.dtype], _rows(scales, "scales"),
        None if zeros is None else zeros.data_ptr(), 0 if zeros is None else _rows(zeros, "zeros"),
        None if bias is None else bias.data_ptr(), group, y.data_ptr(), _rows(y, "out"),
        None if ws is None else ws.data_ptr(), need,
        _get_raw_stream(_get_device()) if stream is None else stream.cuda_stream)
    if status:
        _check(status)


def ck_int4_quantize(w, group: int, qweight, scales, zeros, stream=None):
    """Fills qweight, scales and, unless None (symmetric), zeros from w [V, K]."""
    if w.dtype not in DTYPES or scales.dtype not in DTYPES or not w.is_cuda or w.dim() != 2:
        raise ValueError("w (2-D) and scales are CUDA tensors of float32, bfloat16 or float16")
    if group not in INT4_GROUPS:
        raise ValueError(f"group_size must be one of {INT4_GROUPS}, not {group}")
    V, K = w.shape
    G, dev = -(-K // group), w.get_device()
    _like(qweight, dev, torch.uint8, (V, (K + 1) // 2), "qweight")
    _like(scales, dev, None, (V, G), "scales")
    if zeros is not None:
        _like(zeros, dev, torch.uint8, (V, G), "zeros")
    _check(load().ck_int4_quantize(
        w.data_ptr(), DTYPES[w.dtype], V, K, _rows(w, "w"), group, 1 if zeros is None else 0,
        qweight.data_ptr(), _rows(qweight, "qweight"), scales.data_ptr(), DTYPES[scales.dtype],
        _rows(scales, "scales"), None if zeros is None else zeros.data_ptr(),
        0 if zeros is None else _rows(zeros, "zeros"), _raw_stream(stream)))


def ck_logits_workspace_size(B: int, V: int, L: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ck_logits_workspace_size(B, V, L, ctypes.byref(n)))
    return n.value


def ck_control_logits(call: LogitCall, stream=None):
    status = (_lib or load()).ck_control_logits(
        ctypes.byref(call),
        _get_raw_stream(_get_device()) if stream is None else stream.cuda_stream)
    if status:
        _check(status)


def ck_gated_sizes(T: int, B: int, N: int):
    """(bytes of kept, bytes of workspace)."""
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().ck_gated_sizes(T, B, N, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def ck_gated_forward(call: GatedCall, stream=None):
    _check((_lib or load()).ck_gated_forward(ctypes.byref(call), _raw_stream(stream)))


def ck_gated_backward(call: GatedCall, stream=None):
    _check((_lib or load()).ck_gated_backward(ctypes.byref(call), _raw_stream(stream)))


def gradient_list(grads, outs=None):
    """A ck_gradient array of dense tensors and of where they are clipped to (themselves)."""
    array = (Gradient * len(grads))()
    for g, o, entry in zip(grads, outs or grads, array):
        if g.dtype not in DTYPES or not g.is_cuda or o.dtype != g.dtype or o.numel() != g.numel():
            raise ValueError("gradients are CUDA tensors of float32, bfloat16 or float16, out like them")
        entry.grad, entry.out, entry.n, entry.dtype = g.data_ptr(), o.data_ptr(), g.numel(), DTYPES[g.dtype]
    return array


def ck_clip_workspace_size(array) -> int:
    n = ctypes.c_size_t()
    _check(load().ck_clip_workspace_size(array, len(array), ctypes.byref(n)))
    return n.value


def ck_grad_norm(array, norm, workspace, stream=None):
    _need(norm, torch.float32, "norm")
    _check((_lib or load()).ck_grad_norm(array, len(array), _ptr(norm), _ptr(workspace), workspace.numel() * 8,
                                         _raw_stream(stream)))


def ck_clip_gradients(array, max_norm: float, norm, workspace, stream=None):
    _need(norm, torch.float32, "norm")
    _check((_lib or load()).ck_clip_gradients(array, len(array), float(max_norm), _ptr(norm), _ptr(workspace),
                                              workspace.numel() * 8, _raw_stream(stream)))


def ck_beam_workspace_size(dtype, B: int, K: int, V: int, beams: int) -> int:
    n = ctypes.c_size_t()
    _check(load().ck_beam_workspace_size(DTYPES[dtype], B, K, V, beams, ctypes.byref(n)))
    return n.value


def ck_beam_select(call: BeamCall, stream=None):
    _check((_lib or load()).ck_beam_select(ctypes.byref(call), _raw_stream(stream)))


def ck_reorder_states(array, parents, B: int, K: int, beams: int, stream=None):
    _need(parents, torch.int64, "parents")
    _check((_lib or load()).ck_reorder_states(array, len(array), _ptr(parents), B, K, beams, _raw_stream(stream)))


def ck_forward_static_scratch(handle, edge_values, leak, bias, drives, state0, microsteps,
                              states_out, saved, stream=None):
    for t, n in ((edge_values, "edge_values"), (leak, "leak"), (bias, "bias"),
                 (drives, "drives"), (state0, "state0"), (states_out, "states_out")):
        _need(t, torch.float32, n)
    B = state0.shape[0]
    T = states_out.shape[0]
    _shapes(handle, B, T, edge_values=edge_values, leak=leak, bias=bias, drives=drives,
            state0=state0, states_out=states_out)
    _check(load().ck_forward_static_scratch(
        handle, _ptr(edge_values), _ptr(leak), _ptr(bias),
        _ptr(drives) if drives is not None and drives.numel() else None, _ptr(state0), B, T,
        microsteps, _ptr(states_out), _ptr(saved), saved.numel() * saved.element_size(),
        _stream(stream)))


def ck_query_status(scratch, stream=None):
    _check(load().ck_query_status(_ptr(scratch), _stream(stream)))


def ck_graph_memory(handle):
    """(device bytes, pinned host bytes) the graph handle holds."""
    d, h = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().ck_graph_memory(handle, ctypes.byref(d), ctypes.byref(h)))
    return d.value, h.value


TILING_KEYS = ("C", "G", "P", "max_rows", "max_fin", "max_chunk", "max_edges", "ptr_len")


def ck_graph_tiling(handle, direction: int) -> dict:
    """The shared-memory tiling of one direction (all zero when it has none)."""
    info = (ctypes.c_int64 * 8)()
    _check(load().ck_graph_tiling(handle, direction, info))
    return dict(zip(TILING_KEYS, list(info)))


def ck_graph_export_tiling(handle, direction: int, meta, ptr, col, perm, rowid, stream=None):
    _check(load().ck_graph_export_tiling(handle, direction, _ptr(meta), _ptr(ptr), _ptr(col),
                                         _ptr(perm), _ptr(rowid), _stream(stream)))


def ck_query_status_static(stream=None):
    _check(load().ck_query_status_static(_stream(stream)))


def ck_probe_read(buf, reps, sink, stream=None):
    _check(load().ck_probe_read(_ptr(buf), buf.numel() * buf.element_size(), reps, _ptr(sink),
                                _stream(stream)))


def ck_probe_read_shape(buf, reps, load_bytes, depth, threads, ctas_per_sm, sink, stream=None):
    _check(load().ck_probe_read_shape(_ptr(buf), buf.numel() * buf.element_size(), reps,
                                      load_bytes, depth, threads, ctas_per_sm, _ptr(sink),
                                      _stream(stream)))


def ck_probe_grid_barrier(scheme, ctas, cluster, crossings, rows_per_cta, rows, words, status,
                          stream=None):
    _need(words, torch.int32, "words")
    _need(status, torch.int32, "status")
    if words.numel() < PROBE_BARRIER_WORDS or status.numel() < 1:
        raise ValueError(f"words needs {PROBE_BARRIER_WORDS} elements, status one")
    if rows_per_cta > 0:
        _need(rows, torch.float32, "rows")
        if rows.numel() < ctas * rows_per_cta * 32:
            raise ValueError("rows holds fewer than ctas * rows_per_cta * 32 floats")
    _check(load().ck_probe_grid_barrier(scheme, ctas, cluster, crossings, rows_per_cta,
                                        _ptr(rows) if rows_per_cta > 0 else None, _ptr(words),
                                        _ptr(status), _stream(stream)))


def ck_phase_profile_read(clear: bool = True):
    """The profiling build's phase counters as nested lists
    [direction][CTA][word] of ints (layout in ck.h); raises CKError
    (CK_ERR_UNSUPPORTED) in every other build."""
    n = 2 * PHASE_PROFILE_CTAS * PHASE_PROFILE_WORDS
    buf = (ctypes.c_uint64 * n)()
    _check(load().ck_phase_profile_read(ctypes.cast(buf, ctypes.c_void_p), n, 1 if clear else 0))
    flat = list(buf)
    per = PHASE_PROFILE_CTAS * PHASE_PROFILE_WORDS
    return [[flat[d * per + c * PHASE_PROFILE_WORDS:d * per + (c + 1) * PHASE_PROFILE_WORDS]
             for c in range(PHASE_PROFILE_CTAS)] for d in range(2)]


def ck_probe_gather(rows, idx, sink, stream=None):
    _need(rows, torch.float32, "rows")
    _need(idx, torch.int32, "idx")
    _check(load().ck_probe_gather(_ptr(rows), rows.shape[0], rows.shape[1], _ptr(idx),
                                  idx.numel(), _ptr(sink), _stream(stream)))


def ck_set_option(opt: int, value: int):
    _check(load().ck_set_option(opt, int(value)))


def ck_get_option(opt: int) -> int:
    return int(load().ck_get_option(opt))


def ck_last_launch_count() -> int:
    return int(load().ck_last_launch_count())
