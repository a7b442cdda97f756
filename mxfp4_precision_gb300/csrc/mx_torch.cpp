// mx_torch.cpp -- Python entry points of the operators between the GEMMs over
// the C ABI (include/mx.h): checks and unpacks torch tensors, allocates the
// outputs and passes the current stream.  No arithmetic here.
//
// A CPython module rather than ctypes because these calls are short: a norm of
// one token takes 2.5 us on the GPU, its call through ctypes 20 us on the host
// (half of it four torch.empty), and clipping 64 tensors 65 us (five accessors
// a tensor).
#include <Python.h>

#include <initializer_list>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mx.h"

namespace {

PyObject *g_check = nullptr;  // _binding._check(status, what): raises MXError

// A Python exception is set.
struct Raised {};

template <typename... Args>
[[noreturn]] void refuse(const char *format, Args... args) {
    PyErr_Format(PyExc_ValueError, format, args...);
    throw Raised{};
}

void check(mx_status status, const char *what) {
    if (status == MX_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", static_cast<int>(status), what);
    Py_XDECREF(r);
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a torch.Tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    return t;
}

// Refuses tensors that are not on the device of the call's first: the launch goes
// there, where another device's address may fault or be read before it is written.
void on_device(const at::Tensor &t, const char *name, c10::Device device) {
    if (t.device() != device)
        refuse("%s must be on %s like the call's first tensor, not on %s", name, device.str().c_str(),
               t.device().str().c_str());
}
struct Argument {
    int at;
    const char *name;
};
void on_device(PyObject *const *a, std::initializer_list<Argument> others, c10::Device device) {
    for (const Argument &o : others)
        if (a[o.at] != Py_None) on_device(tensor(a[o.at], o.name), o.name, device);
}

int type_of(const at::Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kBFloat16:
        case at::kShort:
        case at::kUInt16: return MX_TYPE_BF16;
        case at::kFloat: return MX_TYPE_F32;
        default: refuse("%s must be bf16 (torch.bfloat16 or raw 16-bit patterns) or float32", name);
    }
}

// A matrix whose rows are contiguous.
struct Matrix {
    void *p = nullptr;
    int type = 0;
    int64_t pitch = 0;
};

Matrix matrix_of(const at::Tensor &t, const char *name, int64_t rows, int64_t cols) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse("%s must be [%lld, %lld]", name, static_cast<long long>(rows),
               static_cast<long long>(cols));
    if (t.stride(1) != 1 && cols > 1) refuse("%s must have contiguous rows", name);
    return {t.data_ptr(), type_of(t, name), rows > 1 ? t.stride(0) : cols};
}

const at::Tensor &matrix(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2) refuse("%s must be 2-D", name);
    return t;
}

const at::Tensor &vector(PyObject *o, const char *name, int64_t n, int *type) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse("%s must be contiguous and [%lld]", name, static_cast<long long>(n));
    *type = type_of(t, name);
    return t;
}

at::Tensor empty(const at::Tensor &like, at::IntArrayRef sizes, at::ScalarType type) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

PyObject *wrap(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

template <typename... T>
PyObject *tuple_of(const T &...t) {
    PyObject *r = PyTuple_New(sizeof...(t));
    if (r == nullptr) throw Raised{};
    Py_ssize_t i = 0;
    for (PyObject *o : {wrap(t)...}) {
        if (o == nullptr) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Device of the call and its current stream.
struct Here {
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit Here(const at::Tensor &t)
        : guard(t.device()),
          stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
};

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred() != nullptr) throw Raised{};
    return v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred() != nullptr) throw Raised{};
    return static_cast<float>(v);
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// The encoded rows of a [T][K] output; none for MX_FORMAT_NONE.
struct EncodedRows {
    at::Tensor codes, scales;
    int format = MX_FORMAT_NONE;
    void *codes_p = nullptr, *scales_p = nullptr;

    EncodedRows(const at::Tensor &like, PyObject *fmt, int64_t T, int64_t K) {
        if (fmt == Py_None) return;
        format = static_cast<int>(integer(fmt));
        if (format != MX_FORMAT_MXFP4 && format != MX_FORMAT_MXFP8)
            refuse("fmt must be None, FMT_MXFP4 or FMT_MXFP8");
        codes = empty(like, {T, format == MX_FORMAT_MXFP8 ? K : K / 2}, at::kByte);
        scales = empty(like, {std::max<int64_t>(1, mx_scales_bytes(T, K))}, at::kByte);
        codes_p = codes.data_ptr();
        scales_p = scales.data_ptr();
    }
};

// A given workspace, or a new one of `bytes`.
struct Workspace {
    at::Tensor t;
    size_t bytes;
    Workspace(const at::Tensor &like, PyObject *given, size_t need) : bytes(need) {
        if (given == Py_None) {
            t = empty(like, {std::max<int64_t>(1, need)}, at::kByte);
            return;
        }
        t = tensor(given, "workspace");
        if (!t.is_contiguous()) refuse("workspace must be contiguous");
        bytes = t.nbytes();
    }
};

// rmsnorm(x, weight, residual, eps, fmt, want_y, out_h) -> (h, y, codes, scales, rstd)
PyObject *rmsnorm(PyObject *const *a) {
    const at::Tensor &x = matrix(a[0], "x");
    on_device(a, {{1, "weight"}, {2, "residual"}, {6, "out_h"}}, x.device());
    const Here here(x);
    const int64_t T = x.size(0), K = x.size(1);
    const Matrix xm = matrix_of(x, "x", T, K);
    int wt;
    const at::Tensor &w = vector(a[1], "weight", K, &wt);
    at::Tensor h;
    Matrix rm, hm;
    if (a[2] != Py_None) {
        const at::Tensor &r = matrix(a[2], "residual");
        rm = matrix_of(r, "residual", T, K);
        h = a[6] != Py_None ? tensor(a[6], "out_h") : empty(x, {T, K}, r.scalar_type());
        hm = matrix_of(h, "out_h", T, K);
        if (hm.type != rm.type) refuse("out_h must have the residual's type");
    } else if (a[6] != Py_None) {
        refuse("out_h needs a residual");
    }
    at::Tensor y;
    if (truth(a[5])) y = empty(x, {T, K}, at::kBFloat16);
    const EncodedRows e(x, a[4], T, K);
    const at::Tensor rstd = empty(x, {T}, at::kFloat);
    check(mx_rmsnorm(xm.p, xm.type, xm.pitch, rm.p, rm.type, rm.pitch, w.data_ptr(), wt, real(a[3]),
                     T, K, hm.p, hm.pitch, y.defined() ? y.data_ptr() : nullptr, e.format, e.codes_p,
                     e.scales_p, static_cast<float *>(rstd.data_ptr()), here.stream),
          "mx_rmsnorm");
    return tuple_of(h, y, e.codes, e.scales, rstd);
}

// rmsnorm_backward(dy, h, weight, rstd, dres, want_dw, ws, out_dx) -> (dx, dw)
PyObject *rmsnorm_backward(PyObject *const *a) {
    const at::Tensor &dy = matrix(a[0], "dy");
    on_device(a, {{1, "h"}, {2, "weight"}, {3, "rstd"}, {4, "dres"}, {6, "workspace"}, {7, "out_dx"}}, dy.device());
    const Here here(dy);
    const int64_t T = dy.size(0), K = dy.size(1);
    const Matrix dm = matrix_of(dy, "dy", T, K);
    const at::Tensor &h = matrix(a[1], "h");
    const Matrix hm = matrix_of(h, "h", T, K);
    int wt, rt;
    const at::Tensor &w = vector(a[2], "weight", K, &wt), &rstd = vector(a[3], "rstd", T, &rt);
    if (rt != MX_TYPE_F32) refuse("rstd must be float32");
    Matrix gm;
    if (a[4] != Py_None) {
        gm = matrix_of(matrix(a[4], "dres"), "dres", T, K);
        if (gm.type != hm.type) refuse("dres must have h's type");
    }
    const at::Tensor dx = a[7] != Py_None ? tensor(a[7], "out_dx") : empty(dy, {T, K}, h.scalar_type());
    const Matrix om = matrix_of(dx, "out_dx", T, K);
    if (om.type != hm.type) refuse("out_dx must have h's type");
    at::Tensor dw, ws;
    size_t bytes = 0;
    if (truth(a[5])) {
        dw = empty(dy, {K}, at::kFloat);
        Workspace given(dy, a[6], mx_rmsnorm_backward_workspace_bytes(T, K));
        ws = given.t;
        bytes = given.bytes;
    }
    check(mx_rmsnorm_backward(dm.p, dm.type, dm.pitch, hm.p, hm.type, hm.pitch, w.data_ptr(), wt,
                              static_cast<const float *>(rstd.data_ptr()), gm.p, gm.pitch, T, K, om.p,
                              om.pitch, dw.defined() ? static_cast<float *>(dw.data_ptr()) : nullptr,
                              ws.defined() ? ws.data_ptr() : nullptr, bytes, here.stream),
          "mx_rmsnorm_backward");
    return tuple_of(dx, dw);
}

// swiglu(gu, fmt, want_y) -> (y, codes, scales)
PyObject *swiglu(PyObject *const *a) {
    const at::Tensor &gu = matrix(a[0], "gu");
    const Here here(gu);
    const int64_t T = gu.size(0), F = gu.size(1) / 2;
    if (gu.size(1) % 2 != 0) refuse("gu must have an even number of columns");
    const Matrix m = matrix_of(gu, "gu", T, 2 * F);
    at::Tensor y;
    if (truth(a[2])) y = empty(gu, {T, F}, at::kBFloat16);
    const EncodedRows e(gu, a[1], T, F);
    check(mx_swiglu(m.p, m.type, m.pitch, T, F, y.defined() ? y.data_ptr() : nullptr, e.format,
                    e.codes_p, e.scales_p, here.stream),
          "mx_swiglu");
    return tuple_of(y, e.codes, e.scales);
}

// swiglu_backward(dy, gu, out) -> dgu
PyObject *swiglu_backward(PyObject *const *a) {
    const at::Tensor &dy = matrix(a[0], "dy");
    on_device(a, {{1, "gu"}, {2, "out"}}, dy.device());
    const Here here(dy);
    const int64_t T = dy.size(0), F = dy.size(1);
    const Matrix dm = matrix_of(dy, "dy", T, F);
    const Matrix gm = matrix_of(matrix(a[1], "gu"), "gu", T, 2 * F);
    const at::Tensor out = a[2] != Py_None ? tensor(a[2], "out") : empty(dy, {T, 2 * F}, at::kBFloat16);
    const Matrix om = matrix_of(out, "out", T, 2 * F);
    if (om.type != MX_TYPE_BF16 || om.pitch != 2 * F) refuse("out must be bf16 and contiguous");
    check(mx_swiglu_backward(dm.p, dm.type, dm.pitch, gm.p, gm.type, gm.pitch, T, F, om.p, here.stream),
          "mx_swiglu_backward");
    return wrap(out);
}

// The tensors of a Python sequence (none for None): addresses, sizes, types; all on
// the device of the sequence's first, or on the one given.
struct Tensors {
    std::vector<void *> p;
    std::vector<int64_t> n;
    std::vector<int> type;
    at::Tensor first;

    Tensors(PyObject *list, const char *name, const at::Tensor *on = nullptr) {
        if (list == Py_None) return;
        PyObject *s = PySequence_Fast(list, "a sequence of tensors is expected");
        if (s == nullptr) throw Raised{};
        struct Release {
            PyObject *s;
            ~Release() { Py_DECREF(s); }
        } release{s};
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(s);
        p.reserve(count);
        n.reserve(count);
        type.reserve(count);
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(s, i), name);
            if (i == 0) first = t;
            on_device(t, name, (on != nullptr ? *on : first).device());
            if (!t.is_contiguous()) refuse("%s must be contiguous", name);
            p.push_back(t.data_ptr());
            n.push_back(t.numel());
            type.push_back(type_of(t, name));
        }
    }
};

// clip(grads, out, scale, max_norm, eps, ws) -> norm; scale false: the norm alone.
PyObject *clip(PyObject *const *a) {
    const Tensors g(a[0], "gradient");
    const bool scale = truth(a[2]);
    if (g.p.empty()) refuse("no gradients");
    const at::Tensor &like = g.first;
    const Tensors out(a[1], "out", &like);
    on_device(a, {{5, "workspace"}}, like.device());
    const Here here(like);
    const int64_t count = static_cast<int64_t>(g.p.size());
    const at::Tensor norm = empty(like, {1}, at::kFloat);
    const Workspace ws(like, a[5], mx_grad_workspace_bytes(count));
    float *norm_p = static_cast<float *>(norm.data_ptr());
    if (!scale) {
        check(mx_grad_norm(g.p.data(), g.n.data(), g.type.data(), count, norm_p, ws.t.data_ptr(),
                           ws.bytes, here.stream),
              "mx_grad_norm");
    } else if (a[1] == Py_None) {
        check(mx_clip_grads(g.p.data(), g.n.data(), g.type.data(), nullptr, nullptr, count,
                            real(a[3]), real(a[4]), norm_p, ws.t.data_ptr(), ws.bytes, here.stream),
              "mx_clip_grads");
    } else {
        if (out.n != g.n) refuse("out must hold one tensor of the same size for each gradient");
        check(mx_clip_grads(g.p.data(), g.n.data(), g.type.data(), out.p.data(), out.type.data(),
                            count, real(a[3]), real(a[4]), norm_p, ws.t.data_ptr(), ws.bytes,
                            here.stream),
              "mx_clip_grads");
    }
    return wrap(norm);
}

// Argument count, and C++ exceptions turned into Python's (torch's own by its rules).
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_check(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XDECREF(g_check);
    g_check = f;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef g_methods[] = {method<rmsnorm, 7>("rmsnorm"),
                           method<rmsnorm_backward, 8>("rmsnorm_backward"),
                           method<swiglu, 3>("swiglu"),
                           method<swiglu_backward, 3>("swiglu_backward"),
                           method<clip, 6>("clip"),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mx_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mx_torch() { return PyModule_Create(&g_module); }
