// The short way from Python to the operators of a token model, for the calls of an answering
// loop, whose kernels take less time than marshalling a dozen arguments through
// ctypes does.  Each function here checks its arguments, allocates what the call
// returns and calls the library's C entry.  What it does not take (a wrong type or
// shape, another device, a gradient to be recorded, strides that do not join) it
// leaves to the Python form of the same call by returning None, which does it or says
// what is wrong.
//
// It links with no libck: `bind` receives the entries' addresses from the library
// that the process has loaded, whichever variant that is.
#include <Python.h>

#include <cfloat>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck.h"

namespace {

decltype(&ck_dropout) dropout_entry;
decltype(&ck_int4_matvec) matvec_entry;
decltype(&ck_int4_workspace_size) matvec_size_entry;
decltype(&ck_control_logits) logits_entry;
decltype(&ck_logits_workspace_size) logits_size_entry;
decltype(&ck_gated_sizes) gated_size_entry;
decltype(&ck_gated_forward) gated_forward_entry;
decltype(&ck_gated_backward) gated_backward_entry;
decltype(&ck_clip_workspace_size) clip_size_entry;
decltype(&ck_grad_norm) norm_entry;
decltype(&ck_clip_gradients) clip_entry;
decltype(&ck_beam_workspace_size) beam_size_entry;
decltype(&ck_beam_select) beam_entry;
decltype(&ck_reorder_states) reorder_entry;
PyObject *fail_callable;  // raises CKError for a status

PyObject *leave_it() { Py_RETURN_NONE; }

PyObject *raise_status(ck_status st) {
    PyObject *r = PyObject_CallFunction(fail_callable, "i", (int)st);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "an operator failed");
    return nullptr;
}

int dtype_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return CK_F32;
        case at::kBFloat16: return CK_BF16;
        case at::kHalf: return CK_F16;
        default: return -1;
    }
}

// (asked before the device, which a process without one does not have)
bool cuda_tensor(PyObject *o) { return THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(); }

// Whether autograd follows t: it is to get a gradient, or carries a tangent.
// tangents: whether there can be any.
bool followed(const at::Tensor &t, bool tangents) {
    if (!t.unsafeGetTensorImpl()->autograd_meta()) return false;  // (most have none)
    return (t.requires_grad() && c10::GradMode::is_enabled()) || (tangents && t.unsafeGetTensorImpl()->_fw_grad(0, t).defined());
}

// A tensor of a call, on the device `dev`, not followed by autograd, and whose memory holds
// its numbers (a view may be noted as conjugated or negated: those are left).
struct Operand {
    const at::Tensor *t = nullptr;
    bool none = true, good = true;
    Operand(PyObject *o, int dev, bool tangents = true) {
        if (o == Py_None) return;
        none = false;
        good = THPVariable_Check(o);
        if (!good) return;
        t = &THPVariable_Unpack(o);
        good = t->is_cuda() && t->device().index() == dev && t->layout() == at::kStrided && !t->is_conj() && !t->is_neg() &&
               !followed(*t, tangents);
    }
    bool is(at::ScalarType type) const { return t->scalar_type() == type; }
    bool sizes(int64_t a) const { return t->dim() == 1 && t->size(0) == a; }
    bool sizes(int64_t a, int64_t b) const { return t->dim() == 2 && t->size(0) == a && t->size(1) == b; }
};

// Elements between the dense rows of a 2-D tensor; -1 where they are not dense.
int64_t row_stride(const at::Tensor &t) {
    const int64_t n = t.size(0), m = t.size(1);
    if (m > 1 && t.stride(1) != 1) return -1;
    return n > 1 ? t.stride(0) : m;
}

bool whole_number(PyObject *o, uint64_t &v) {
    if (!PyLong_Check(o)) return false;
    v = PyLong_AsUnsignedLongLongMask(o);
    return !(v == (uint64_t)-1 && PyErr_Occurred());
}

// A step: a whole number, or one int64 on the device.
bool step_of(PyObject *o, int dev, uint64_t &step, const int64_t *&at_dev) {
    step = 0;
    at_dev = nullptr;
    if (PyLong_Check(o)) return whole_number(o, step);
    const Operand s(o, dev);
    if (s.none || !s.good || !s.is(at::kLong) || s.t->numel() != 1) return false;
    at_dev = s.t->const_data_ptr<int64_t>();
    return true;
}

// Raises the version of a tensor that a call is about to write, for those who saved it.
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// dropout(x, p, seed, step, locked)
PyObject *dropout(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 5 || !cuda_tensor(a[0]) || !PyFloat_Check(a[1])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand x(a[0], dev);
        uint64_t seed, step;
        const int64_t *step_dev;
        if (!x.good || !whole_number(a[2], seed) || !step_of(a[3], dev, step, step_dev)) {
            PyErr_Clear();
            return leave_it();
        }
        const int dtype = dtype_of(*x.t), dims = (int)x.t->dim();
        const bool locked = a[4] == Py_True;
        if (dtype < 0 || (!locked && a[4] != Py_False) || (locked && dims < 2) || dims > 8) return leave_it();
        // the axes that are left when those that follow one another in memory are joined;
        // a locked mask's repeats stay an axis of their own
        int64_t size[3] = {1, 1, 1}, stride[3] = {0, 0, 0};
        if (x.t->is_contiguous()) {
            const int64_t all = x.t->numel(), first = locked ? x.t->size(0) : 1;
            size[0] = first;
            size[2] = first ? all / first : 0;
            stride[0] = locked ? size[2] : 0;
            stride[2] = 1;
        } else {
            int64_t js[8], jt[8];
            int joined = 0;
            for (int i = locked; i < dims; ++i) {
                const int64_t s = x.t->size(i), t = x.t->stride(i);
                if (s == 1) continue;
                if (joined && jt[joined - 1] == t * s) {
                    js[joined - 1] *= s;
                    jt[joined - 1] = t;
                } else {
                    js[joined] = s;
                    jt[joined++] = t;
                }
            }
            if (joined + locked > 3) return leave_it();
            for (int i = 0; i < joined; ++i) size[3 - joined + i] = js[i], stride[3 - joined + i] = jt[i];
            if (locked) size[0] = x.t->size(0), stride[0] = x.t->stride(0);
        }
        at::Tensor y = at::empty(x.t->sizes(), x.t->options().requires_grad(false), at::MemoryFormat::Contiguous);
        const ck_status st = dropout_entry(x.t->const_data_ptr(), y.data_ptr(), dtype, size[0], size[1], size[2],
                                           stride[0], stride[1], stride[2], size[1] * size[2], size[2], 1, locked,
                                           PyFloat_AS_DOUBLE(a[1]), seed, step, step_dev, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        return THPVariable_Wrap(std::move(y));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// int4_matvec(x, qweight, scales, zeros, bias, group, out)
PyObject *int4_matvec(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 7 || !cuda_tensor(a[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand x(a[0], dev), q(a[1], dev), s(a[2], dev), z(a[3], dev), b(a[4], dev), o(a[6], dev);
        uint64_t group;
        if (!x.good || q.none || !q.good || s.none || !s.good || !z.good || !b.good || !o.good ||
            !whole_number(a[5], group) || (group != 32 && group != 64 && group != 128)) {
            PyErr_Clear();
            return leave_it();
        }
        const int dtype = dtype_of(*x.t), scale_dtype = dtype_of(*s.t);
        if (dtype < 0 || scale_dtype < 0 || x.t->dim() != 2 || q.t->dim() != 2 || x.t->size(1) < 1) return leave_it();
        const int64_t M = x.t->size(0), K = x.t->size(1), V = q.t->size(0), G = (K + (int64_t)group - 1) / (int64_t)group;
        if (!q.is(at::kByte) || q.t->size(1) != (K + 1) / 2 || !s.sizes(V, G) ||
            (!z.none && (!z.is(at::kByte) || !z.sizes(V, G))) ||
            (!b.none && (!b.is(at::kFloat) || !b.sizes(V) || !b.t->is_contiguous())) ||
            (!o.none && (o.t->scalar_type() != x.t->scalar_type() || !o.sizes(M, V))))
            return leave_it();
        const int64_t xs = row_stride(*x.t), qs = row_stride(*q.t), ss = row_stride(*s.t),
                      zs = z.none ? 0 : row_stride(*z.t), os = o.none ? V : row_stride(*o.t);
        if (xs < 0 || qs < 0 || ss < 0 || zs < 0 || os < 0) return leave_it();
        if (V > 1 && qs % 16 && qs == q.t->size(1)) return leave_it();  // rows to be laid out first
        const int64_t pitch = V > 1 ? qs : (q.t->size(1) + 15) / 16 * 16;
        size_t need = 0;
        ck_status st = matvec_size_entry(dtype, M, K, V, (int64_t)group, &need);
        if (st != CK_OK) return raise_status(st);
        at::Tensor y = o.none ? at::empty({M, V}, x.t->options().requires_grad(false)) : *o.t, ws;
        if (need) ws = at::empty({(int64_t)need}, q.t->options());
        if (!o.none) written(y);
        st = matvec_entry(x.t->const_data_ptr(), dtype, M, K, xs, (const uint8_t *)q.t->const_data_ptr(), V, pitch,
                          s.t->const_data_ptr(), scale_dtype, ss, z.none ? nullptr : (const uint8_t *)z.t->const_data_ptr(),
                          zs, b.none ? nullptr : (const float *)b.t->const_data_ptr(), (int64_t)group, y.data_ptr(), os,
                          need ? ws.data_ptr() : nullptr, need, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        return THPVariable_Wrap(std::move(y));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// control(logits, history, history_len, prompt_len, repetition, frequency, presence,
// bias, mask, temperature, out, give, seed, step); out: None, a tensor or True (a new
// one); give: 0 the logits, 1 the tokens, 2 both
PyObject *control(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 14 || !cuda_tensor(a[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand x(a[0], dev), text(a[1], dev), bias(a[7], dev), mask(a[8], dev);
        if (!x.good || !text.good || !bias.good || !mask.good || x.t->dim() != 2) return leave_it();
        ck_logit_call c{};
        const int64_t B = x.t->size(0), V = x.t->size(1);
        c.logits = x.t->const_data_ptr();
        c.dtype = dtype_of(*x.t);
        c.B = B;
        c.V = V;
        c.logits_stride = row_stride(*x.t);
        if (c.dtype < 0 || c.logits_stride < 0) return leave_it();
        if (!text.none) {
            if ((!text.is(at::kLong) && !text.is(at::kInt)) || text.t->dim() != 2 || text.t->size(0) != B) return leave_it();
            c.history = text.t->const_data_ptr();
            c.history_bits = text.is(at::kLong) ? 64 : 32;
            c.L = text.t->size(1);
            c.history_stride = row_stride(*text.t);
            if (c.history_stride < 0) return leave_it();
        }
        const void **length[2] = {&c.history_len, &c.prompt_len};
        for (int i = 0; i < 2; ++i) {
            const Operand l(a[2 + i], dev);
            if (l.none) continue;
            if (text.none || !l.good || l.t->scalar_type() != text.t->scalar_type() || !l.sizes(B) || !l.t->is_contiguous())
                return leave_it();
            *length[i] = l.t->const_data_ptr();
        }
        const struct {
            int arg;
            const float **row;
            float *all, usual;
            double least;
        } per_row[4] = {{4, &c.repetition, &c.repetition_all, 1.f, 1e-30},
                        {5, &c.frequency, &c.frequency_all, 0.f, -1e30},
                        {6, &c.presence, &c.presence_all, 0.f, -1e30},
                        {9, &c.temperature, &c.temperature_all, 1.f, 0.0}};
        for (const auto &r : per_row) {
            PyObject *o = a[r.arg];
            *r.all = r.usual;
            if (o == Py_None) continue;
            if (PyFloat_Check(o)) {
                const double v = PyFloat_AS_DOUBLE(o);
                if (!(v >= r.least && v <= FLT_MAX) || (v != 0 && fabs(v) < FLT_MIN)) return leave_it();
                *r.all = (float)v;
                continue;
            }
            const Operand t(o, dev);
            if (!t.good || !t.is(at::kFloat) || !t.sizes(B) || !t.t->is_contiguous()) return leave_it();
            *r.row = t.t->const_data_ptr<float>();
        }
        auto per_token = [&](const Operand &t, at::ScalarType type, int64_t m, const void **at, int64_t *stride) {
            if (t.none) return true;
            if (!t.is(type) || (!t.sizes(B, m) && !t.sizes(m))) return false;
            if (m > 1 && t.t->stride(t.t->dim() - 1) != 1) return false;
            *at = t.t->const_data_ptr();
            *stride = t.t->dim() == 2 ? t.t->stride(0) : 0;
            return true;
        };
        const void *bias_at = nullptr, *mask_at = nullptr;
        if (!per_token(bias, at::kFloat, V, &bias_at, &c.bias_stride) ||
            !per_token(mask, at::kInt, (V + 31) / 32, &mask_at, &c.mask_stride))
            return leave_it();
        c.bias = (const float *)bias_at;
        c.mask = (const int32_t *)mask_at;
        const long give = PyLong_AsLong(a[11]);
        at::Tensor out, tokens, ws;
        if (a[10] == Py_True) {
            out = at::empty(x.t->sizes(), x.t->options().requires_grad(false), at::MemoryFormat::Contiguous);
        } else if (a[10] != Py_None) {
            const Operand o(a[10], dev);
            if (!o.good || o.t->scalar_type() != x.t->scalar_type() || !o.sizes(B, V)) return leave_it();
            out = *o.t;
        }
        if (out.defined()) {
            c.out = out.data_ptr();
            c.out_stride = row_stride(out);
            if (c.out_stride < 0) return leave_it();
        }
        if (give > 0) {
            if (a[12] != Py_None) {
                uint64_t seed, step;
                if (!whole_number(a[12], seed) || !step_of(a[13], dev, step, c.step_dev)) {
                    PyErr_Clear();
                    return leave_it();
                }
                c.sample = 1;
                c.seed = seed;
                c.step = step;
            }
            size_t need = 0;
            const ck_status st = V < 1 ? CK_OK : logits_size_entry(B, V, c.L, &need);
            if (st != CK_OK) return raise_status(st);
            const auto whole = x.t->options().dtype(at::kLong).requires_grad(false);
            tokens = at::empty({B}, whole);
            c.tokens = tokens.data_ptr<int64_t>();
            if (need) {
                ws = at::empty({(int64_t)(need / 8)}, whole);
                c.workspace = ws.data_ptr();
                c.workspace_bytes = (int64_t)need;
            }
        }
        if (a[10] != Py_True && out.defined()) written(out);
        const ck_status st = logits_entry(&c, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        if (give == 0) return THPVariable_Wrap(std::move(out));
        if (give == 1) return THPVariable_Wrap(std::move(tokens));
        PyObject *pair = PyTuple_New(2);
        if (!pair) return nullptr;
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(tokens)));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(out)));
        return pair;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// A tuple of tensors, None for those that are not defined.
PyObject *tuple_of(std::initializer_list<at::Tensor> list) {
    PyObject *r = PyTuple_New((Py_ssize_t)list.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &t : list) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// A workspace on the current device and stream, without a tensor around it.
struct Space {
    void *at = nullptr;
    explicit Space(size_t bytes) {
        if (bytes) at = c10::cuda::CUDACachingAllocator::raw_alloc(bytes);
    }
    ~Space() {
        if (at) c10::cuda::CUDACachingAllocator::raw_delete(at);
    }
    Space(const Space &) = delete;
    Space &operator=(const Space &) = delete;
};

// (without the dispatcher's way to the same function)
at::Tensor empty_like_type(at::IntArrayRef sizes, const at::Tensor &like, at::ScalarType type) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

// The operands that both directions of a gated recurrence take.
bool gated_operands(ck_gated_call &c, const Operand &x, const Operand &gate, const Operand &lengths, PyObject *form) {
    if (x.none || !x.good || gate.none || !gate.good || !lengths.good || x.t->dim() != 3 || !PyUnicode_Check(form)) return false;
    c.dtype = dtype_of(*x.t);
    if (c.dtype < 0 || gate.t->scalar_type() != x.t->scalar_type() || gate.t->sizes() != x.t->sizes()) return false;
    if (PyUnicode_CompareWithASCIIString(form, "leak") == 0)
        c.form = CK_GATED_LEAK;
    else if (PyUnicode_CompareWithASCIIString(form, "decay") == 0)
        c.form = CK_GATED_DECAY;
    else
        return false;
    c.T = x.t->size(0), c.B = x.t->size(1), c.N = x.t->size(2);
    if (c.N > 1 && (x.t->stride(2) != 1 || gate.t->stride(2) != 1)) return false;
    c.x = x.t->const_data_ptr(), c.gate = gate.t->const_data_ptr();
    c.x_step = x.t->stride(0), c.x_row = x.t->stride(1);
    c.gate_step = gate.t->stride(0), c.gate_row = gate.t->stride(1);
    if (!lengths.none) {
        if (!lengths.is(at::kLong) || !lengths.sizes(c.B) || !lengths.t->is_contiguous()) return false;
        c.lengths = lengths.t->const_data_ptr<int64_t>();
    }
    return true;
}

bool state_operand(const float *&at, const Operand &s, int64_t B, int64_t N) {
    at = nullptr;
    if (s.none) return true;
    if (!s.good || !s.is(at::kFloat) || !s.sizes(B, N) || !s.t->is_contiguous()) return false;
    at = s.t->const_data_ptr<float>();
    return true;
}

// gated(x, gate, state0, lengths, form, keep): (out, state, kept or None)
PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 6 || !cuda_tensor(a[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand x(a[0], dev), gate(a[1], dev), state0(a[2], dev), lengths(a[3], dev);
        ck_gated_call c{};
        if (!gated_operands(c, x, gate, lengths, a[4]) || !state_operand(c.state0, state0, c.B, c.N)) return leave_it();
        size_t kept_bytes = 0, need = 0;
        ck_status st = gated_size_entry(c.T, c.B, c.N, &kept_bytes, &need);
        if (st != CK_OK) return raise_status(st);
        at::Tensor out = empty_like_type({c.T, c.B, c.N}, *x.t, x.t->scalar_type());
        at::Tensor state = empty_like_type({c.B, c.N}, *x.t, at::kFloat), kept;
        c.out = out.data_ptr();
        c.state = state.data_ptr<float>();
        if (a[5] == Py_True) {
            kept = empty_like_type({(int64_t)(kept_bytes / 4)}, *x.t, at::kFloat);
            c.kept = kept.data_ptr<float>();
        }
        const Space ws(need);
        c.workspace = ws.at;
        c.workspace_bytes = (int64_t)need;
        st = gated_forward_entry(&c, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        return tuple_of({out, state, kept});
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// gated_backward(x, gate, kept, d_out, d_state, lengths, form, want_x, want_gate, want_state0)
PyObject *gated_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 10 || !cuda_tensor(a[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand x(a[0], dev), gate(a[1], dev), kept(a[2], dev), d(a[3], dev), ds(a[4], dev), lengths(a[5], dev);
        ck_gated_call c{};
        if (!gated_operands(c, x, gate, lengths, a[6]) || !state_operand(c.d_state, ds, c.B, c.N)) return leave_it();
        size_t kept_bytes = 0, need = 0;
        ck_status st = gated_size_entry(c.T, c.B, c.N, &kept_bytes, &need);
        if (st != CK_OK) return raise_status(st);
        if (kept.none || !kept.good || !kept.is(at::kFloat) || kept.t->numel() * 4 != (int64_t)kept_bytes || !kept.t->is_contiguous())
            return leave_it();
        c.kept = const_cast<float *>(kept.t->const_data_ptr<float>());  // the backward reads it
        if (!d.none) {
            if (!d.good || d.t->scalar_type() != x.t->scalar_type() || d.t->sizes() != x.t->sizes() || (c.N > 1 && d.t->stride(2) != 1))
                return leave_it();
            c.d_out = d.t->const_data_ptr();
            c.d_out_step = d.t->stride(0), c.d_out_row = d.t->stride(1);
        }
        at::Tensor dx, dgate, dstate0;
        if (a[7] == Py_True) {
            dx = empty_like_type({c.T, c.B, c.N}, *x.t, x.t->scalar_type());
            c.dx = dx.data_ptr();
        }
        if (a[8] == Py_True) {
            dgate = empty_like_type({c.T, c.B, c.N}, *x.t, x.t->scalar_type());
            c.dgate = dgate.data_ptr();
        }
        if (a[9] == Py_True) {
            dstate0 = empty_like_type({c.B, c.N}, *x.t, at::kFloat);
            c.d_state0 = dstate0.data_ptr<float>();
        }
        const Space ws(need);
        c.workspace = ws.at;
        c.workspace_bytes = (int64_t)need;
        st = gated_backward_entry(&c, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        return tuple_of({dx, dgate, dstate0});
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

bool list_of(PyObject *o) { return PyList_CheckExact(o) || PyTuple_CheckExact(o); }

// clip(grads, max_norm, out): the norm of a list of tensors; max_norm None: no clipping;
// out None: in place
PyObject *clip(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 3 || !list_of(a[0]) || (a[2] != Py_None && !list_of(a[2]))) return leave_it();
        const bool clips = a[1] != Py_None, apart = a[2] != Py_None;
        if (clips && !PyFloat_Check(a[1])) return leave_it();
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
        if (count < 1 || (apart && PySequence_Fast_GET_SIZE(a[2]) != count)) return leave_it();
        PyObject **in = PySequence_Fast_ITEMS(a[0]), **to = apart ? PySequence_Fast_ITEMS(a[2]) : in;
        if (!cuda_tensor(in[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        std::vector<ck_gradient> list((size_t)count);
        std::vector<const at::Tensor *> outs((size_t)count);
        // (asked once: a view's tangent is looked for in its base)
        const bool tangents = torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const Operand g(in[i], dev, tangents);
            if (g.none || !g.good || !g.t->is_contiguous()) return leave_it();
            list[i].grad = g.t->const_data_ptr();
            list[i].n = g.t->numel();
            list[i].dtype = dtype_of(*g.t);
            if (list[i].dtype < 0) return leave_it();
            outs[i] = g.t;
            if (apart) {
                const Operand o(to[i], dev, tangents);
                if (o.none || !o.good || !o.t->is_contiguous() || o.t->scalar_type() != g.t->scalar_type() || o.t->sizes() != g.t->sizes())
                    return leave_it();
                outs[i] = o.t;
            }
            if (clips) list[i].out = outs[i]->data_ptr();
        }
        at::Tensor norm = empty_like_type({}, *outs[0], at::kFloat);
        const auto call = [&](size_t bytes) {
            const Space ws(bytes);
            return clips ? clip_entry(list.data(), count, PyFloat_AS_DOUBLE(a[1]), norm.data_ptr<float>(), ws.at, (int64_t)bytes, stream_of(dev))
                         : norm_entry(list.data(), count, norm.data_ptr<float>(), ws.at, (int64_t)bytes, stream_of(dev));
        };
        // (enough for any list of some thousand tensors; asked for where it is not)
        ck_status st = call(1 << 16);
        if (st == CK_ERR_WORKSPACE) {
            size_t need = 0;
            st = clip_size_entry(list.data(), count, &need);
            if (st == CK_OK) st = call(need);
        }
        if (st != CK_OK) return raise_status(st);
        if (clips)
            for (const at::Tensor *o : outs) written(*o);
        return THPVariable_Wrap(std::move(norm));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// beam(logits, scores, ended, end_token, beams): (scores, parents, tokens, ended)
PyObject *beam(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 5 || !cuda_tensor(a[0])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand z(a[0], dev), s(a[1], dev), e(a[2], dev);
        if (!z.good || s.none || !s.good || !e.good || z.t->dim() != 3) return leave_it();
        ck_beam_call c{};
        c.dtype = dtype_of(*z.t);
        c.B = z.t->size(0), c.K = z.t->size(1), c.V = z.t->size(2);
        c.beams = c.K;
        c.end_token = -1;
        uint64_t v;
        if (a[3] != Py_None) {
            if (!whole_number(a[3], v) || v >= (uint64_t)c.V) {
                PyErr_Clear();
                return leave_it();
            }
            c.end_token = (int64_t)v;
        }
        if (a[4] != Py_None) {
            if (!whole_number(a[4], v) || v < 1 || v > 64) {
                PyErr_Clear();
                return leave_it();
            }
            c.beams = (int64_t)v;
        }
        if (c.dtype < 0 || c.K < 1 || c.V < 1 || (c.V > 1 && z.t->stride(2) != 1) || !s.is(at::kFloat) || !s.sizes(c.B, c.K) ||
            !s.t->is_contiguous())
            return leave_it();
        if (!e.none) {
            if (!e.is(at::kBool) || !e.sizes(c.B, c.K) || !e.t->is_contiguous() || c.end_token < 0) return leave_it();
            c.ended = (const uint8_t *)e.t->const_data_ptr();
        }
        c.logits = z.t->const_data_ptr();
        c.logits_row = z.t->stride(0), c.logits_beam = z.t->stride(1);
        c.scores = s.t->const_data_ptr<float>();
        size_t need = 0;
        ck_status st = beam_size_entry(c.dtype, c.B, c.K, c.V, c.beams, &need);
        if (st != CK_OK) return raise_status(st);
        at::Tensor scores = empty_like_type({c.B, c.beams}, *z.t, at::kFloat);
        at::Tensor parents = empty_like_type({c.B, c.beams}, *z.t, at::kLong);
        at::Tensor tokens = empty_like_type({c.B, c.beams}, *z.t, at::kLong);
        at::Tensor over = empty_like_type({c.B, c.beams}, *z.t, at::kBool);
        const Space ws(need);
        c.scores_out = scores.data_ptr<float>();
        c.parents = parents.data_ptr<int64_t>(), c.tokens = tokens.data_ptr<int64_t>();
        c.ended_out = (uint8_t *)over.data_ptr();
        c.workspace = ws.at;
        c.workspace_bytes = (int64_t)need;
        st = beam_entry(&c, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        return tuple_of({scores, parents, tokens, over});
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Whether t[b][k] is a dense row.
bool rows_inside(const at::Tensor &t) {
    int64_t at = 1;
    for (int64_t i = t.dim() - 1; i > 1; --i) {
        if (t.size(i) != 1 && t.stride(i) != at) return false;
        at *= t.size(i);
    }
    return true;
}

// reorder(states, parents, out): a list of tensors; out None: new ones
PyObject *reorder(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != 3 || !list_of(a[0]) || (a[2] != Py_None && !list_of(a[2])) || !cuda_tensor(a[1])) return leave_it();
        const int dev = c10::cuda::current_device();
        const Operand p(a[1], dev);
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
        const bool apart = a[2] != Py_None;
        if (!p.good || !p.is(at::kLong) || p.t->dim() != 2 || !p.t->is_contiguous() || count < 1 ||
            (apart && PySequence_Fast_GET_SIZE(a[2]) != count))
            return leave_it();
        PyObject **in = PySequence_Fast_ITEMS(a[0]), **to = apart ? PySequence_Fast_ITEMS(a[2]) : nullptr;
        const int64_t B = p.t->size(0), beams = p.t->size(1);
        int64_t K = 0;
        std::vector<ck_beam_state> list((size_t)count);
        std::vector<at::Tensor> outs((size_t)count);
        if (B < 1) return leave_it();
        // all are looked at before any is made or written
        for (Py_ssize_t i = 0; i < count; ++i) {
            const Operand s(in[i], dev);
            if (s.none || !s.good || s.t->dim() < 2 || s.t->size(0) != B || !rows_inside(*s.t)) return leave_it();
            if (i == 0) K = s.t->size(1);
            if (s.t->size(1) != K || K < 1) return leave_it();
            if (apart) {
                const Operand o(to[i], dev);
                if (o.none || !o.good || o.t->scalar_type() != s.t->scalar_type() || o.t->dim() != s.t->dim() || o.t->size(0) != B ||
                    o.t->size(1) != beams || o.t->sizes().slice(2) != s.t->sizes().slice(2) || !rows_inside(*o.t))
                    return leave_it();
                outs[i] = *o.t;
            }
        }
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor &s = THPVariable_Unpack(in[i]);
            if (!apart) {
                c10::SmallVector<int64_t, 8> shape(s.sizes().begin(), s.sizes().end());
                shape[1] = beams;
                outs[i] = empty_like_type(shape, s, s.scalar_type());
            }
            const int64_t size = (int64_t)s.element_size();
            ck_beam_state &e = list[i];
            e.in = s.const_data_ptr();
            e.out = outs[i].data_ptr();
            e.bytes = s.numel() / (B * K) * size;
            e.in_row = s.stride(0) * size, e.in_beam = s.stride(1) * size;
            e.out_row = outs[i].stride(0) * size, e.out_beam = outs[i].stride(1) * size;
        }
        const ck_status st = reorder_entry(list.data(), count, p.t->const_data_ptr<int64_t>(), B, K, beams, stream_of(dev));
        if (st != CK_OK) return raise_status(st);
        PyObject *r = PyList_New(count);
        if (!r) return nullptr;
        for (Py_ssize_t i = 0; i < count; ++i) {
            if (apart) written(outs[i]);
            PyObject *o = apart ? Py_NewRef(to[i]) : THPVariable_Wrap(outs[i]);
            if (!o) {
                Py_DECREF(r);
                return nullptr;
            }
            PyList_SET_ITEM(r, i, o);
        }
        return r;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(addresses, fail): the library's entries, in the order below, and what raises an
// error for a status
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *list, *fail;
    if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &list, &fail)) return nullptr;
    void **entries[] = {(void **)&dropout_entry, (void **)&matvec_entry, (void **)&matvec_size_entry, (void **)&logits_entry,
                        (void **)&logits_size_entry, (void **)&gated_size_entry, (void **)&gated_forward_entry,
                        (void **)&gated_backward_entry, (void **)&clip_size_entry, (void **)&norm_entry, (void **)&clip_entry,
                        (void **)&beam_size_entry, (void **)&beam_entry, (void **)&reorder_entry};
    constexpr Py_ssize_t kEntries = sizeof(entries) / sizeof(entries[0]);
    if (PyTuple_GET_SIZE(list) != kEntries) {
        PyErr_SetString(PyExc_ValueError, "bind takes an address for each entry");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < kEntries; ++i) {
        void *at = PyLong_AsVoidPtr(PyTuple_GET_ITEM(list, i));
        if (!at && PyErr_Occurred()) return nullptr;
        *entries[i] = at;
    }
    Py_INCREF(fail);
    Py_XSETREF(fail_callable, fail);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"dropout", (PyCFunction)(void (*)(void))dropout, METH_FASTCALL, nullptr},
    {"int4_matvec", (PyCFunction)(void (*)(void))int4_matvec, METH_FASTCALL, nullptr},
    {"control", (PyCFunction)(void (*)(void))control, METH_FASTCALL, nullptr},
    {"gated", (PyCFunction)(void (*)(void))gated, METH_FASTCALL, nullptr},
    {"gated_backward", (PyCFunction)(void (*)(void))gated_backward, METH_FASTCALL, nullptr},
    {"clip", (PyCFunction)(void (*)(void))clip, METH_FASTCALL, nullptr},
    {"beam", (PyCFunction)(void (*)(void))beam, METH_FASTCALL, nullptr},
    {"reorder", (PyCFunction)(void (*)(void))reorder, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ck_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ck_binding() { return PyModule_Create(&module); }
