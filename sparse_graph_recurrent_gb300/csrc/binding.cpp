// The short way from Python to the readout operators, for the calls of an answering
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

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck.h"

namespace {

decltype(&ck_dropout) dropout_entry;
decltype(&ck_int4_matvec) matvec_entry;
decltype(&ck_int4_workspace_size) matvec_size_entry;
decltype(&ck_control_logits) logits_entry;
decltype(&ck_logits_workspace_size) logits_size_entry;
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
bool followed(const at::Tensor &t) {
    return (t.requires_grad() && c10::GradMode::is_enabled()) || t.unsafeGetTensorImpl()->_fw_grad(0, t).defined();
}

// A tensor of a call, on the device `dev` and not followed by autograd.
struct Operand {
    const at::Tensor *t = nullptr;
    bool none = true, good = true;
    Operand(PyObject *o, int dev) {
        if (o == Py_None) return;
        none = false;
        good = THPVariable_Check(o);
        if (!good) return;
        t = &THPVariable_Unpack(o);
        good = t->is_cuda() && t->device().index() == dev && t->layout() == at::kStrided && !followed(*t);
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

// bind(dropout, int4_matvec, int4_workspace_size, control_logits, logits_workspace_size,
// fail): addresses of the library's entries, and what raises an error for a status
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long at[5];
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KKKKKO", &at[0], &at[1], &at[2], &at[3], &at[4], &fail)) return nullptr;
    dropout_entry = (decltype(dropout_entry))at[0];
    matvec_entry = (decltype(matvec_entry))at[1];
    matvec_size_entry = (decltype(matvec_size_entry))at[2];
    logits_entry = (decltype(logits_entry))at[3];
    logits_size_entry = (decltype(logits_size_entry))at[4];
    Py_INCREF(fail);
    Py_XSETREF(fail_callable, fail);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"dropout", (PyCFunction)(void (*)(void))dropout, METH_FASTCALL, nullptr},
    {"int4_matvec", (PyCFunction)(void (*)(void))int4_matvec, METH_FASTCALL, nullptr},
    {"control", (PyCFunction)(void (*)(void))control, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ck_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ck_binding() { return PyModule_Create(&module); }
