"""Readout operators without a GPU: the oracle's generator against the published
known answers, the view logic of dropout, and refusals made on the host."""
import ctypes

import numpy as np
import pytest
import torch

import readout_oracle as ro


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_oracle_generator_gives_the_published_answers(ctr, key, want):
    # the block's index is counter words 0 and 1; an element index is four times it, so
    # blocks above 2^62 are reached through the words directly
    block, step = ctr[0] | ctr[1] << 32, ctr[2] | ctr[3] << 32
    if block < 1 << 62:
        got = ro.philox_words(np.arange(4, dtype=np.uint64) + np.uint64(4 * block),
                              key[0] | key[1] << 32, step)
    else:
        c = list(ctr)
        k = list(key)
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & ro.M32, (a >> 32) ^ c[3] ^ k[1], a & ro.M32]
            k = [(k[0] + 0x9E3779B9) & ro.M32, (k[1] + 0xBB67AE85) & ro.M32]
        got = c
    assert [int(v) for v in got] == list(want)


@pytest.mark.parametrize("locked", [False, True])
@pytest.mark.parametrize("make", [
    lambda b: b[:6 * 4 * 5].view(6, 4, 5),
    lambda b: b[:6 * 4 * 9].view(6, 4, 9)[..., :5],
    lambda b: b[:6 * 4 * 5].view(4, 6, 5).transpose(0, 1),
    lambda b: b[:6 * 4 * 5].view(5, 4, 6).permute(2, 1, 0),
    lambda b: b[:5].view(1, 1, 5).expand(6, 4, 5),
    lambda b: b[:2 * 3 * 4 * 10].view(2, 3, 4, 10)[:, :, 1:3, ::2],
    lambda b: b[:240].view(3, 2, 2, 20)[:, :, ::2].permute(0, 3, 1, 2),
    lambda b: b[:1].view(1, 1),
    lambda b: b[:40].view(4, 10)[:, ::3],
])
def test_views_join_into_three_axes(make, locked):
    """The sizes and strides name the same elements, in the same order, as the tensor."""
    from sparse_graph_recurrent_gb300.readout import _as3
    x = make(torch.arange(1000))
    y, n, s = _as3(x, locked)
    got = torch.as_strided(y, n, s, y.storage_offset())
    assert torch.equal(got.reshape(-1), x.reshape(-1))
    if locked:
        assert n[0] == x.shape[0]


def _lib():
    from sparse_graph_recurrent_gb300 import _ck
    return _ck, _ck.load()


def test_dropout_refuses_on_the_host():
    _, lib = _lib()
    buf = (ctypes.c_float * 8)()

    def call(dtype=0, n=(1, 1, 8), p=0.5, x=buf, y=buf):
        return lib.ck_dropout(x, y, dtype, *n, 0, 0, 1, 0, 0, 1, 0, p, 1, 1, None, None)

    assert call(dtype=3) == 1 and call(dtype=-1) == 1
    for p in (-0.1, 1.0001, float("nan"), float("inf")):
        assert call(p=p) == 1
        assert b"p must" in lib.ck_last_error_message()
    assert call(n=(1, -1, 8)) == 1
    assert call(x=None) == 1 and call(y=None) == 1
    assert call(n=(1 << 40, 1 << 40, 1)) == 7
    assert call(n=(0, 4, 8)) == 0 and call(n=(4, 0, 8), x=None, y=None) == 0  # nothing to do


def test_int4_refuses_on_the_host():
    _, lib = _lib()
    raw = ctypes.create_string_buffer(4096)
    base = -(-ctypes.addressof(raw) // 16) * 16

    def call(x=base, dtype=0, M=1, K=64, xs=64, q=base, V=2, pitch=32, s=base, sdt=0, ss=2, z=None,
             zs=0, group=32, y=base, ys=2):
        return lib.ck_int4_matvec(x, dtype, M, K, xs, q, V, pitch, s, sdt, ss, z, zs, None, group, y,
                                  ys, None, 0, None)

    assert call(dtype=5) == 1 and call(sdt=9) == 1
    for g in (0, 16, 33, 256, -32):
        assert call(group=g) == 1
    assert call(K=0) == 1 and call(M=-1) == 1 and call(V=-1) == 1
    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1 and call(y=None) == 1
    assert call(pitch=40) == 1 and call(q=base + 8) == 1 and call(pitch=16) == 1
    assert b"16 bytes" in lib.ck_last_error_message()
    assert call(ss=1) == 1 and call(ys=1) == 1 and call(z=base, zs=1) == 1
    assert call(K=1 << 30) == 7
    assert call(M=0) == 0 and call(V=0) == 0
    assert lib.ck_int4_quantize(base, 0, 2, 64, 64, 48, 1, base, 32, base, 0, 2, None, 0, None) == 1
    assert lib.ck_int4_quantize(base, 0, 2, 64, 64, 32, 0, base, 32, base, 0, 2, None, 0, None) == 1
    assert lib.ck_int4_quantize(base, 0, 2, 64, 64, 32, 1, base, 31, base, 0, 2, None, 0, None) == 1
    assert lib.ck_int4_quantize(base, 0, 0, 64, 64, 32, 1, base, 32, base, 0, 2, None, 0, None) == 0


def test_control_logits_refuses_on_the_host():
    _ck, lib = _lib()
    buf = (ctypes.c_float * 8)()
    at = ctypes.addressof(buf)

    def call(**kw):
        args = dict(logits=at, dtype=0, B=1, V=8, logits_stride=8, out=at, out_stride=8,
                    repetition_all=1.0, temperature_all=1.0)
        args.update(kw)
        return lib.ck_control_logits(ctypes.byref(_ck.LogitCall(**args)), None)

    assert lib.ck_control_logits(None, None) == 1
    assert call(dtype=4) == 1 and call(V=0) == 1 and call(B=-1) == 1
    assert call(logits=None) == 1 and call(out=None) == 1
    assert call(history=at, history_bits=16, L=4) == 1 and call(history=at, history_bits=32, L=-1) == 1
    assert call(V=1 << 31) == 7 and call(B=1 << 17) == 7
    assert call(B=0) == 0


def test_struct_matches_the_header():
    """ck_logit_call's fields, in order, are the binding's."""
    import os
    import re

    from sparse_graph_recurrent_gb300 import _ck
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "ck.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} ck_logit_call;", text).group(1)
    kinds = {"int64_t": ctypes.c_int64, "uint64_t": ctypes.c_uint64, "float": ctypes.c_float}
    want = []
    for line in body.split(";"):
        m = re.match(r"\s*((?:const )?\w+)\s+(.*)", line.strip(), flags=re.S)
        if not m:
            continue
        for name in m.group(2).split(","):
            name = name.strip()
            kind = ctypes.c_void_p if name.startswith("*") else kinds[m.group(1)]
            want.append((name.lstrip("*"), kind))
    assert want == [(n, k) for n, k in _ck.LogitCall._fields_]


def test_cpu_tensors_are_refused():
    import sparse_graph_recurrent_gb300 as ck
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        ck.dropout(x, 0.5, 1)
    with pytest.raises(ValueError):
        ck.int4_quantize(x)
    with pytest.raises(ValueError):
        ck.int4_matvec(x, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1))
    with pytest.raises(ValueError):
        ck.control_logits(x)
    with pytest.raises(ValueError):
        ck.pick_tokens(x)


def test_the_compiled_module_leaves_cpu_tensors():
    from sparse_graph_recurrent_gb300 import _ck
    x = torch.zeros(2, 64)
    assert _ck.native().dropout(x, 0.5, 1, 0, False) is None
    assert _ck.native().int4_matvec(x, x, x, None, None, 32, None) is None
    assert _ck.native().control(x, *[None] * 9, True, 0, None, 0) is None


def test_workspace_comes_from_the_stream_that_uses_it(monkeypatch):
    """A product on a named stream allocates on that stream: a block of the current one may
    still be written by kernels that are pending there."""
    from contextlib import contextmanager

    from sparse_graph_recurrent_gb300 import _ck

    class Cuda:
        """As much of a CUDA tensor as the call looks at."""
        is_cuda, device = True, torch.device("cuda", 0)

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

        dim = lambda self: len(self.shape)  # noqa: E731
        stride = lambda self, i=None: (self.shape[1], 1) if i is None else (self.shape[1], 1)[i]  # noqa: E731
        get_device = lambda self: 0  # noqa: E731
        data_ptr = lambda self: 4096  # noqa: E731
        record_stream = lambda self, stream: None  # noqa: E731

    class Stream:
        cuda_stream = 77

    at, took, ran = [0], [], []

    @contextmanager
    def stream(s):
        at.append(s.cuda_stream)
        yield
        at.pop()

    def empty(*size, **kw):
        took.append(at[-1])
        return Cuda(torch.uint8, *size)

    class Lib:
        @staticmethod
        def ck_int4_matvec(*a):
            ran.append(a[-1])
            return 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(_ck, "_lib", Lib)
    monkeypatch.setattr(_ck, "_get_device", lambda: 0)
    monkeypatch.setattr(_ck, "_get_raw_stream", lambda device: 0)
    monkeypatch.setattr(_ck, "_int4_ws", {(0, torch.float32, 2, 64, 8, 32): 4096})
    args = (Cuda(torch.float32, 2, 64), Cuda(torch.uint8, 8, 32), Cuda(torch.float32, 8, 2), None, None, 32,
            Cuda(torch.float32, 2, 8))
    _ck.ck_int4_matvec(*args)
    _ck.ck_int4_matvec(*args, stream=Stream())
    assert ran == [0, 77] and took == [0, 77]


def test_the_library_loads_without_the_compiled_module(monkeypatch):
    """No host compiler for Python modules: the library loads, says so once, and every call
    is left to its Python form."""
    import sparse_graph_recurrent_gb300 as ck
    from sparse_graph_recurrent_gb300 import _ck

    def fails(force=False):
        raise RuntimeError("g++ failed")

    _ck.load()
    monkeypatch.setattr(_ck, "_lib", None)
    monkeypatch.setattr(_ck, "_native", None)
    monkeypatch.setattr(_ck._build, "build_binding", fails)
    with pytest.warns(RuntimeWarning, match="g\\+\\+ failed"):
        lib = _ck.load()
    assert lib is _ck.load() and lib.ck_query_status is not None
    x = torch.zeros(2, 64)
    assert _ck.native().dropout(x, 0.5, 1, 0, False) is None
    assert _ck.native().int4_matvec(x, x, x, None, None, 32, None) is None
    assert _ck.native().control(x, *[None] * 9, True, 0, None, 0) is None
    for call in (lambda: ck.dropout(x, 0.5, 1), lambda: ck.control_logits(x), lambda: ck.pick_tokens(x)):
        with pytest.raises(ValueError):
            call()


def test_a_library_that_does_not_load_is_not_half_loaded(monkeypatch):
    from sparse_graph_recurrent_gb300 import _ck

    def fails(lib):
        raise RuntimeError("no")

    _ck.load()
    monkeypatch.setattr(_ck, "_lib", None)
    monkeypatch.setattr(_ck, "_native", None)
    monkeypatch.setattr(_ck, "_load_native", fails)
    for _ in range(2):
        with pytest.raises(RuntimeError):
            _ck.load()


def test_the_compiled_module_is_of_one_interpreter(monkeypatch):
    """Another interpreter or torch has a file of its own; a current one is taken as it is."""
    import sysconfig

    from sparse_graph_recurrent_gb300 import build
    here = build.build_binding()
    assert sysconfig.get_config_var("EXT_SUFFIX") in here and torch.__version__ in here
    monkeypatch.setattr(build.subprocess, "run", None)  # nothing is compiled again
    assert build.build_binding() == here
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".other.so" if name == "EXT_SUFFIX" else real(name))
    assert build.binding_path() != here


def test_weight_rows_are_laid_out_again():
    import sparse_graph_recurrent_gb300 as ck
    q = torch.randint(0, 256, (7, 33), dtype=torch.uint8)
    a = ck.int4_rows(q)
    assert torch.equal(a, q) and a.stride() == (48, 1) and a.data_ptr() % 16 == 0
    assert ck.int4_rows(a) is a and ck.int4_rows(a[2:5]).data_ptr() == a[2:].data_ptr()
    for v in (q.t().contiguous().t(), a[:, 1:], q[:1], q[:0]):
        assert torch.equal(ck.int4_rows(v), v)
    for bad in (q.int(), q[0]):
        with pytest.raises(ValueError):
            ck.int4_rows(bad)


def test_misaligned_pointers_are_refused_on_the_host():
    """Each pointer, off by a byte, is an error and not a misaligned access on the device."""
    _ck, lib = _lib()
    raw = ctypes.create_string_buffer(8192)
    base = -(-ctypes.addressof(raw) // 64) * 64

    def refused(status):
        return status == 1 and b"not aligned" in lib.ck_last_error_message()

    for dtype in (0, 1, 2):
        for off in ("x", "y", "step"):
            a = {k: base + (off == k) for k in ("x", "y", "step")}
            assert refused(lib.ck_dropout(a["x"], a["y"], dtype, 1, 1, 8, 0, 0, 1, 0, 0, 1, 0, 0.5, 1, 1, a["step"], None))
        for off in ("x", "s", "b", "y"):
            a = {k: base + (off == k) for k in ("x", "s", "b", "y")}
            assert refused(lib.ck_int4_matvec(a["x"], dtype, 1, 64, 64, base, 2, 32, a["s"], dtype, 2, None, 0, a["b"], 32,
                                              a["y"], 2, None, 0, None))
        for off in ("w", "s"):
            a = {k: base + (off == k) for k in ("w", "s")}
            assert refused(lib.ck_int4_quantize(a["w"], dtype, 2, 64, 64, 32, 1, base, 32, a["s"], dtype, 2, None, 0, None))
        for bits in (32, 64):
            for off in ("logits", "out", "tokens", "step_dev", "history", "history_len", "prompt_len", "repetition",
                        "frequency", "presence", "temperature", "bias", "mask"):
                a = dict(dtype=dtype, B=1, V=8, logits_stride=8, out_stride=8, repetition_all=1.0, temperature_all=1.0,
                         logits=base, out=base, history=base, history_bits=bits, L=4, history_stride=4)
                a[off] = base + 1
                assert refused(lib.ck_control_logits(ctypes.byref(_ck.LogitCall(**a)), None)), off


def test_rows_of_out_that_overlap_are_refused():
    """Several rows written to one place would leave whichever came last."""
    _ck, lib = _lib()
    buf = (ctypes.c_float * 64)()
    for stride in (0, 7, -8):
        a = dict(logits=ctypes.addressof(buf), dtype=0, B=2, V=8, logits_stride=8, out=ctypes.addressof(buf), out_stride=stride,
                 repetition_all=1.0, temperature_all=1.0)
        assert lib.ck_control_logits(ctypes.byref(_ck.LogitCall(**a)), None) == 1
        assert b"overlap" in lib.ck_last_error_message()


def test_a_dropout_output_that_shares_places_is_refused():
    _, lib = _lib()
    buf = (ctypes.c_float * 64)()
    for y in ((0, 8, 1), (8, 0, 1), (16, 8, 0)):
        assert lib.ck_dropout(buf, buf, 0, 2, 2, 2, 0, 0, 0, *y, 0, 0.5, 1, 1, None, None) == 1
        assert b"share a place" in lib.ck_last_error_message()
