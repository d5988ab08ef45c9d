// bind.cpp — the binding of the operators without a psi: torch tensors to disco_tensor views, outputs and
// workspaces that the caller did not give, torch's current stream, a status to an exception.
//
// A call on little data costs the host's time alone, and a call on many gradients the host's time per tensor;
// this module takes 1.5 us a call and 0.03 us a tensor beside the launches where the same marshalling in Python
// took 5 and 0.4.  It holds no arithmetic and no argument checks but the ones a view needs.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

#include "disco.h"

namespace {

PyObject *g_error = nullptr;    // DiscoError(status, message)
PyObject *g_stream = nullptr;   // device index -> the current stream's handle

struct Raised {};   // a Python exception is set

disco_dtype code_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return DISCO_F32;
    case at::kBFloat16: return DISCO_BF16;
    case at::kHalf: return DISCO_F16;
    case at::kFloat8_e4m3fn: return DISCO_F8_E4M3;
    case at::kFloat8_e5m2: return DISCO_F8_E5M2;
    case at::kChar: return DISCO_I8;
    default: return (disco_dtype)99;  // refused by the library
    }
}

const at::Tensor &tensor_of(PyObject *o)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

// A tensor that the caller holds was written: autograd's check of the tensors it saved sees that, as after any
// operation in place.
void wrote(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An argument that may be None.
struct Arg {
    at::Tensor t;
    disco_tensor d = {};
    bool given = false;
    bool callers = false;   // else made here
    Arg() = default;
    explicit Arg(PyObject *o)
    {
        if (o == Py_None) return;
        set(tensor_of(o));
        callers = true;
    }
    void set(const at::Tensor &v)
    {
        if (!v.is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "disco tensors must be contiguous");
            throw Raised();
        }
        t = v;
        given = true;
        d.data = v.data_ptr();
        d.dtype = code_of(v.scalar_type());
        d.ndim = (int32_t)v.dim();
        for (int64_t i = 0; i < v.dim() && i < 5; ++i) d.shape[i] = v.size(i);
    }
    disco_tensor *ptr() { return given ? &d : nullptr; }
    // The tensor handed back, after a call that wrote it.
    PyObject *out() const
    {
        if (callers) wrote(t);
        return THPVariable_Wrap(t);
    }
};

struct Required : Arg {
    explicit Required(PyObject *o) { set(tensor_of(o)); }
};

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

long long whole(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int axis_of(PyObject *o)
{
    const long long v = whole(o);
    return v < -100 || v > 100 ? 100 : (int)v;  // the library refuses both
}

void *stream_of(const at::Tensor &t)
{
    if (!t.is_cuda()) return nullptr;  // the library refuses host memory
    PyObject *i = PyLong_FromLong(t.get_device());
    PyObject *s = i ? PyObject_CallOneArg(g_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!s) throw Raised();
    void *p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
}

[[noreturn]] void raise_status(disco_status st, const char *message)
{
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, message);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

void check(disco_status st)
{
    if (st != DISCO_OK) raise_status(st, disco_last_error());
}

// Runs a library call without the interpreter lock.
template <typename F>
void call(F f)
{
    disco_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    check(st);
}

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised &) {
    } catch (...) {  // torch's own, as the exceptions that its users know (out of memory among them)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject *pair(PyObject *a, PyObject *b)
{
    PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

at::Tensor bytes_on(const at::Tensor &like, size_t n)
{
    return at::empty({(int64_t)(n ? n : 1)}, like.options().dtype(at::kByte));
}

// rms_norm(x, w, residual, axis, eps, y, h)
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        Required x(a[0]), w(a[1]);
        Arg r(a[2]), y(a[5]), h(a[6]);
        const int axis = axis_of(a[3]);
        const float eps = (float)real(a[4]);
        if (!y.given) y.set(at::empty_like(x.t));
        if (r.given && !h.given) h.set(at::empty_like(x.t));
        void *s = stream_of(x.t);
        call([&] { return disco_rms_norm(&x.d, r.ptr(), &w.d, axis, eps, &y.d, h.ptr(), s); });
        return r.given ? pair(y.out(), h.out()) : y.out();
    });
}

// rms_norm_f8(x, w, residual, axis, eps, group, e5m2, q, scale, h)
PyObject *rms_norm_f8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        Required x(a[0]), w(a[1]);
        Arg r(a[2]), q(a[7]), scale(a[8]), h(a[9]);
        const int axis = axis_of(a[3]);
        const float eps = (float)real(a[4]);
        const int64_t group = whole(a[5]);
        if (!q.given) q.set(at::empty_like(x.t, x.t.options().dtype(whole(a[6]) ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn)));
        if (!scale.given) {
            auto shape = x.t.sizes().vec();
            const int64_t i = axis < 0 ? axis + x.t.dim() : axis;
            if (i >= 0 && i < x.t.dim())  // else the library refuses the axis
                shape[i] = group > 0 ? (shape[i] + group - 1) / group : 1;
            scale.set(at::empty(shape, x.t.options().dtype(at::kFloat)));
        }
        if (r.given && !h.given) h.set(at::empty_like(x.t));
        void *s = stream_of(x.t);
        call([&] { return disco_rms_norm_f8(&x.d, r.ptr(), &w.d, axis, eps, group, &q.d, &scale.d, h.ptr(), s); });
        if (!r.given) return pair(q.out(), scale.out());
        PyObject *o[3] = {q.out(), scale.out(), h.out()};
        PyObject *t = o[0] && o[1] && o[2] ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
        for (PyObject *v : o) Py_XDECREF(v);
        return t;
    });
}

// dequantize(q, scale, code of the output's type or -1, axis, group, out)
PyObject *dequantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        Required q(a[0]), scale(a[1]);
        Arg out(a[5]);
        const int axis = axis_of(a[3]);
        const int64_t group = whole(a[4]);
        if (!out.given) {
            const long long code = whole(a[2]);
            out.set(at::empty_like(q.t, q.t.options().dtype(code == DISCO_F32 ? at::kFloat : code == DISCO_F16 ? at::kHalf : at::kBFloat16)));
        }
        void *s = stream_of(q.t);
        call([&] { return disco_dequantize(&q.d, &scale.d, axis, group, &out.d, s); });
        return out.out();
    });
}

// rms_norm_bwd(h, w, gy, gh, axis, eps, gx, dw, workspace)
PyObject *rms_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        Required h(a[0]), w(a[1]), gy(a[2]);
        Arg gh(a[3]), gx(a[6]), dw(a[7]), ws(a[8]);
        const int axis = axis_of(a[4]);
        const float eps = (float)real(a[5]);
        if (!gx.given) gx.set(at::empty_like(h.t));
        if (!dw.given) dw.set(at::empty_like(w.t));
        if (!ws.given) {
            size_t need = 0;
            check(disco_rms_norm_bwd_workspace(&h.d, axis, &need));
            ws.set(bytes_on(h.t, need));
        }
        void *s = stream_of(h.t);
        call([&] {
            return disco_rms_norm_bwd(&h.d, &w.d, &gy.d, gh.ptr(), axis, eps, &gx.d, &dw.d, ws.d.data, ws.t.nbytes(), s);
        });
        return pair(gx.out(), dw.out());
    });
}

// A sequence of tensors as a tuple of its own, which holds them for the call (the sequence is the caller's, and another
// thread or the code of another argument may change it meanwhile), each seen as its elements in a row.
struct List {
    PyObject *seq;
    std::vector<disco_tensor> d;
    explicit List(PyObject *o) : seq(PySequence_Tuple(o))
    {
        if (!seq) throw Raised();
        try {
            d.resize((size_t)PyTuple_GET_SIZE(seq));
            for (int64_t i = 0; i < size(); ++i) {
                const at::Tensor &t = tensor_of(PyTuple_GET_ITEM(seq, i));
                if (!t.is_contiguous()) {
                    PyErr_SetString(PyExc_ValueError, "disco tensors must be contiguous");
                    throw Raised();
                }
                disco_tensor &v = d[(size_t)i];
                v.data = t.data_ptr();
                v.dtype = code_of(t.scalar_type());
                v.ndim = 1;
                v.shape[0] = t.numel();
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
    }
    ~List() { Py_DECREF(seq); }
    List(const List &) = delete;
    int64_t size() const { return (int64_t)d.size(); }
    const at::Tensor &operator[](int64_t i) const { return THPVariable_Unpack(PyTuple_GET_ITEM(seq, i)); }
};

// grad_norm(grads, norm or None) and clip_grads(grads, max_norm, eps, out or None, norm or None): the result's
// tensor is made beside the first gradient where it is not given.
PyObject *grads_call(PyObject *list, PyObject *result, bool clip, float max_norm, float eps, PyObject *into)
{
    List g(list);
    Arg norm(result);
    if (!norm.given) {
        if (g.size() == 0) {
            PyErr_SetString(PyExc_ValueError, "the norm of no tensors needs a device");
            throw Raised();
        }
        norm.set(at::empty({}, g[0].options().dtype(at::kFloat).requires_grad(false)));
    }
    size_t need = 0;
    check(disco_grad_norm_workspace(g.size(), g.d.data(), &need));
    const at::Tensor ws = bytes_on(norm.t, need);
    void *s = stream_of(norm.t);
    const List *written = nullptr;
    std::optional<List> o;
    if (!clip) {
        call([&] { return disco_grad_norm(g.size(), g.d.data(), &norm.d, ws.data_ptr(), need, s); });
    } else if (into == Py_None) {
        call([&] { return disco_clip_grads(g.size(), g.d.data(), max_norm, eps, g.d.data(), &norm.d, ws.data_ptr(), need, s); });
        written = &g;
    } else {
        o.emplace(into);
        if (o->size() != g.size()) {
            PyErr_SetString(PyExc_ValueError, "out must have one tensor for each gradient");
            throw Raised();
        }
        for (int64_t i = 0; i < g.size(); ++i)  // the library sees them as their elements in a row
            if (g[i].sizes() != (*o)[i].sizes())
                raise_status(DISCO_ERR_SHAPE, ("out[" + std::to_string(i) + "] does not have the shape of its gradient").c_str());
        call([&] { return disco_clip_grads(g.size(), g.d.data(), max_norm, eps, o->d.data(), &norm.d, ws.data_ptr(), need, s); });
        written = &*o;
    }
    if (written)
        for (int64_t i = 0; i < written->size(); ++i) wrote((*written)[i]);
    return norm.out();
}

PyObject *grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 2, [&] { return grads_call(a[0], a[1], false, 0.0f, 0.0f, Py_None); });
}

PyObject *clip_grads(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 5, [&] { return grads_call(a[0], a[4], true, (float)real(a[1]), (float)real(a[2]), a[3]); });
}

// ---- channel products in 8-bit integers

at::ScalarType type_of(long long code) { return code == DISCO_F32 ? at::kFloat : code == DISCO_F16 ? at::kHalf : at::kBFloat16; }

// The points of a dense tensor: its shape without the channel axis.  An axis that is out of range takes nothing away (the
// library refuses it).
std::vector<int64_t> points_of(const at::Tensor &x, int axis)
{
    auto shape = x.sizes().vec();
    const int64_t i = axis < 0 ? axis + x.dim() : axis;
    if (i >= 0 && i < x.dim()) shape.erase(shape.begin() + i);
    return shape;
}

// The form of a dense tensor, made where it is not given.
void make_form(const at::Tensor &x, int axis, Arg *q, Arg *scale)
{
    const int64_t i = axis < 0 ? axis + x.dim() : axis;
    const int64_t D = i >= 0 && i < x.dim() ? x.size(i) : 1;
    auto shape = points_of(x, axis);
    if (!scale->given) scale->set(at::empty(shape, x.options().dtype(at::kFloat).requires_grad(false)));
    if (q->given) return;
    shape.push_back((D + 15) / 16 * 16);
    q->set(at::empty(shape, x.options().dtype(at::kChar).requires_grad(false)));
}

// The dense tensor of a form's points with `D` channels at `axis`.
at::Tensor dense_of(const at::Tensor &q, long long D, int axis, at::ScalarType type)
{
    auto shape = q.sizes().vec();
    if (!shape.empty()) shape.pop_back();
    const int64_t i = axis < 0 ? axis + (int64_t)shape.size() + 1 : axis;
    shape.insert(shape.begin() + (i >= 0 && i <= (int64_t)shape.size() ? i : (int64_t)shape.size()), D < 0 ? 0 : D);
    return at::empty(shape, q.options().dtype(type));
}

// quantize_i8(x, act, keep, axis, q, scale, kept, kept_scale)
PyObject *quantize_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject * {
        Required x(a[0]);
        Arg q(a[4]), scale(a[5]), kept(a[6]), ks(a[7]);
        const long long act = whole(a[1]);
        const int keep = PyObject_IsTrue(a[2]), axis = axis_of(a[3]);
        if (keep < 0) throw Raised();
        make_form(x.t, axis, &q, &scale);
        if (keep) make_form(x.t, axis, &kept, &ks);
        void *s = stream_of(x.t);
        call([&] { return disco_quantize_i8(&x.d, (disco_act)act, axis, &q.d, &scale.d, kept.ptr(), ks.ptr(), s); });
        if (!kept.given) return pair(q.out(), scale.out());
        PyObject *o[4] = {q.out(), scale.out(), kept.out(), ks.out()};
        PyObject *t = o[0] && o[1] && o[2] && o[3] ? PyTuple_Pack(4, o[0], o[1], o[2], o[3]) : nullptr;
        for (PyObject *v : o) Py_XDECREF(v);
        return t;
    });
}

// dequantize_i8(q, scale, channels or -1, code of the output's type, axis, out)
PyObject *dequantize_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        Required q(a[0]), scale(a[1]);
        Arg out(a[5]);
        const int axis = axis_of(a[4]);
        if (!out.given) {
            const long long D = whole(a[2]);
            out.set(dense_of(q.t, D < 0 && q.t.dim() ? q.t.size(-1) : D, axis, type_of(whole(a[3]))));
        }
        void *s = stream_of(q.t);
        call([&] { return disco_dequantize_i8(&q.d, &scale.d, axis, &out.d, s); });
        return out.out();
    });
}

// linear_i8(q, scale, w, wscale, bias, code of the output's type, axis, out)
PyObject *linear_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        Required q(a[0]), scale(a[1]), w(a[2]), wscale(a[3]);
        Arg bias(a[4]), y(a[7]);
        const int axis = axis_of(a[6]);
        if (!y.given) y.set(dense_of(q.t, w.t.dim() ? w.t.size(0) : 0, axis, type_of(whole(a[5]))));
        void *s = stream_of(q.t);
        call([&] { return disco_linear_i8(&q.d, &scale.d, &w.d, &wscale.d, bias.ptr(), axis, &y.d, s); });
        return y.out();
    });
}

// linear_i8_bwd_input(gy, w, wscale, channels or -1, act, kept, kept_scale, axis, gx)
PyObject *linear_i8_bwd_input(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        Required gy(a[0]), w(a[1]), wscale(a[2]);
        Arg kept(a[5]), ks(a[6]), gx(a[8]);
        const long long act = whole(a[4]);
        const int axis = axis_of(a[7]);
        if (!gx.given) {
            const long long D = whole(a[3]);
            auto shape = gy.t.sizes().vec();
            const int64_t i = axis < 0 ? axis + gy.t.dim() : axis;
            if (i >= 0 && i < gy.t.dim()) shape[i] = D >= 0 ? D : w.t.dim() ? w.t.size(-1) : 0;
            gx.set(at::empty(shape, gy.t.options()));
        }
        void *s = stream_of(gy.t);
        call([&] { return disco_linear_i8_bwd_input(&gy.d, &w.d, &wscale.d, (disco_act)act, kept.ptr(), ks.ptr(), axis, &gx.d, s); });
        return gx.out();
    });
}

// linear_i8_bwd_weight(gy, q, scale, channels or -1, bias, axis, dw, db, workspace)
PyObject *linear_i8_bwd_weight(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject * {
        Required gy(a[0]), q(a[1]), scale(a[2]);
        Arg dw(a[6]), db(a[7]), ws(a[8]);
        const int bias = PyObject_IsTrue(a[4]), axis = axis_of(a[5]);
        if (bias < 0) throw Raised();
        const int64_t i = axis < 0 ? axis + gy.t.dim() : axis;
        const int64_t Co = i >= 0 && i < gy.t.dim() ? gy.t.size(i) : 1;
        if (!dw.given) {
            const long long D = whole(a[3]);
            dw.set(at::empty({Co, D >= 0 ? D : q.t.dim() ? q.t.size(-1) : 0}, gy.t.options()));
        }
        if (bias && !db.given) db.set(at::empty({Co}, gy.t.options()));
        if (!ws.given) {
            size_t need = 0;
            check(disco_linear_i8_bwd_weight_workspace(&gy.d, axis, dw.t.dim() ? dw.t.size(-1) : 0, db.given, &need));
            if (need) ws.set(bytes_on(gy.t, need));
        }
        void *s = stream_of(gy.t);
        call([&] {
            return disco_linear_i8_bwd_weight(&gy.d, &q.d, &scale.d, axis, &dw.d, db.ptr(), ws.given ? ws.d.data : nullptr,
                                              ws.given ? ws.t.nbytes() : 0, s);
        });
        return db.given ? pair(dw.out(), db.out()) : dw.out();
    });
}

// linear_i8_bwd_weight_workspace(gy, channels, bias, axis)
PyObject *linear_i8_bwd_weight_workspace(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 4, [&]() -> PyObject * {
        Required gy(a[0]);
        const long long C = whole(a[1]);
        const int bias = PyObject_IsTrue(a[2]), axis = axis_of(a[3]);
        if (bias < 0) throw Raised();
        size_t need = 0;
        check(disco_linear_i8_bwd_weight_workspace(&gy.d, axis, C, bias, &need));
        return PyLong_FromSize_t(need);
    });
}

// setup(DiscoError, device index -> current stream)
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 2, [&]() -> PyObject * {
        Py_INCREF(a[0]);
        Py_INCREF(a[1]);
        Py_XDECREF(g_error);
        Py_XDECREF(g_stream);
        g_error = a[0];
        g_stream = a[1];
        Py_RETURN_NONE;
    });
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(setup), FAST(rms_norm), FAST(rms_norm_f8), FAST(dequantize), FAST(rms_norm_bwd),
                           FAST(grad_norm), FAST(clip_grads), FAST(quantize_i8), FAST(dequantize_i8), FAST(linear_i8),
                           FAST(linear_i8_bwd_input), FAST(linear_i8_bwd_weight), FAST(linear_i8_bwd_weight_workspace), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_disco_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__disco_bind(void) { return PyModule_Create(&g_module); }
