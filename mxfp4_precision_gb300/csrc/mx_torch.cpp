// mx_torch.cpp -- Python entry points of the operators between the GEMMs, of the
// products with an epilogue and of those by expert over the C ABI (include/mx.h): checks and unpacks torch tensors, allocates the
// outputs and passes the current stream.  No arithmetic here.
//
// A CPython module rather than ctypes because these calls are short: a norm of
// one token takes 2.5 us on the GPU, its call through ctypes 20 us on the host
// (half of it four torch.empty), and clipping 64 tensors 65 us (five accessors
// a tensor).
#include <Python.h>

#include <algorithm>
#include <array>
#include <initializer_list>
#include <vector>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
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

// Whether somebody looks at what a call allocates: a dispatch mode, the profiler, torch's fill of fresh
// memory in deterministic runs.  Asked once a call (50 ns); a mode's own code may make calls in between.
struct Watched {
    static thread_local bool now;
    const bool before = now;
    Watched() {
        const at::Context &torch = at::globalContext();
        now = c10::impl::tls_is_dispatch_key_included(c10::DispatchKey::Python) || at::hasCallbacks() ||
              (torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory());
    }
    ~Watched() { now = before; }
};
thread_local bool Watched::now = false;

// Without the dispatcher, which takes 0.5 us of a call with two outputs, unless it is watched.
at::Tensor empty(const at::Tensor &like, at::IntArrayRef sizes, at::ScalarType type) {
    if (Watched::now) return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// Contiguous tensors of one type that share one allocation, each at a multiple of 16 bytes.
template <size_t N>
struct Parts {
    std::array<at::Tensor, N> t;
    Parts(const at::Tensor &like, at::ScalarType type, const std::array<std::vector<int64_t>, N> &sizes) {
        const int64_t unit = 16 / static_cast<int64_t>(c10::elementSize(type));
        std::array<int64_t, N> first;
        int64_t all = 0;
        for (size_t i = 0; i < N; ++i) {
            first[i] = all;
            all += (c10::multiply_integers(sizes[i]) + unit - 1) / unit * unit;
        }
        const at::Tensor whole = empty(like, {all}, type);
        for (size_t i = 0; i < N; ++i) {
            t[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
            t[i].unsafeGetTensorImpl()->set_storage_offset(first[i]);
            t[i].unsafeGetTensorImpl()->set_sizes_contiguous(sizes[i]);
        }
    }
};

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
    Watched watched;
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
// 64 bits as they are: a seed may be a negative number or one from 2^63 on.
uint64_t bits(PyObject *o) {
    const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
    if (v == static_cast<uint64_t>(-1) && PyErr_Occurred() != nullptr) throw Raised{};
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

// ---- products with an epilogue, and by expert

// An operand's codes or scales: contiguous bytes, `need` of them at least.
void *bytes_of(PyObject *o, const char *name, size_t need) {
    const at::Tensor &t = tensor(o, name);
    if (t.element_size() != 1 || !t.is_contiguous()) refuse("%s must be contiguous and of 8-bit elements", name);
    if (t.nbytes() < need)
        refuse("%s must hold %llu bytes, not %llu", name, static_cast<unsigned long long>(need),
               static_cast<unsigned long long>(t.nbytes()));
    return t.data_ptr();
}
int operands_of(PyObject *o) {
    const int64_t f = integer(o);
    if (f != MX_FORMAT_MXFP4 && f != MX_FORMAT_MXFP8) refuse("operands must be FMT_MXFP4 or FMT_MXFP8");
    return static_cast<int>(f);
}
size_t codes_need(int operands, int64_t lines, int64_t k) {
    return operands == MX_FORMAT_MXFP8 ? mx_mxfp8_codes_bytes(lines, k) : mx_codes_bytes(lines, k);
}
// The codes and scales at a[0..3] of A ([a_lines], k) and B (`matrices` of [b_lines], k).
struct Operands {
    int format;
    void *aq, *as, *bq, *bs;
    Operands(PyObject *const *a, PyObject *fmt, int64_t a_lines, int64_t matrices, int64_t b_lines, int64_t k)
        : format(operands_of(fmt)) {
        if (a_lines < 0 || b_lines < 0 || k < 0) refuse("sizes must not be negative");
        aq = bytes_of(a[0], "Aq", codes_need(format, a_lines, k));
        as = bytes_of(a[1], "As", mx_scales_bytes(a_lines, k));
        bq = bytes_of(a[2], "Bq", matrices * codes_need(format, b_lines, k));
        bs = bytes_of(a[3], "Bs", matrices * mx_scales_bytes(b_lines, k));
    }
};

// A contiguous int32 tensor of one of a plan's parts.
int32_t *part_of(PyObject *o, const char *name, int64_t *n = nullptr, int64_t want = -1) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kInt || !t.is_contiguous()) refuse("%s must be contiguous and int32", name);
    if (want >= 0 && t.numel() != want) refuse("%s must have %lld elements", name, static_cast<long long>(want));
    if (n != nullptr) *n = t.numel();
    return static_cast<int32_t *>(t.data_ptr());
}
// The plan's tensors at a[0..3]: offsets, counts, slot, source.
struct Plan {
    int32_t *offsets, *counts, *slot, *source;
    int64_t experts, rows, T, picks;
    explicit Plan(PyObject *const *a) {
        int64_t n;
        offsets = part_of(a[0], "plan.offsets", &n);
        experts = n - 1;
        if (experts < 1) refuse("plan.offsets must have an element more than there are experts");
        counts = part_of(a[1], "plan.counts", nullptr, experts);
        slot = part_of(a[2], "plan.slot");
        const at::Tensor &s = THPVariable_Unpack(a[2]);
        if (s.dim() != 2) refuse("plan.slot must be [tokens, choices]");
        T = s.size(0), picks = s.size(1);
        source = part_of(a[3], "plan.source", &rows);
        if (rows % 128 != 0) refuse("plan.source must have a multiple of 128 elements");
    }
};

at::ScalarType out_type(PyObject *f32) { return truth(f32) ? at::kFloat : at::kBFloat16; }

// Bias of `matrices` times [N]; none for None.
void *bias_of(PyObject *o, int64_t matrices, int64_t N, int *type) {
    *type = MX_TYPE_BF16;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "bias");
    const bool shaped = matrices == 0 ? t.dim() == 1 && t.size(0) == N
                                      : t.dim() == 2 && t.size(0) == matrices && t.size(1) == N;
    if (!shaped || !t.is_contiguous())
        refuse(matrices == 0 ? "bias must be contiguous and [N]" : "bias must be contiguous and [experts, N]");
    *type = type_of(t, "bias");
    return t.data_ptr();
}

// gemm_bias_act(Aq, As, Bq, Bs, M, N, K, bias, act, residual, f32, want_y, want_z, fmt, operands, out) -> (y, z, codes, scales)
PyObject *gemm_bias_act(PyObject *const *a) {
    const at::Tensor &like = tensor(a[0], "Aq");
    on_device(a, {{1, "As"}, {2, "Bq"}, {3, "Bs"}, {7, "bias"}, {9, "residual"}, {15, "out"}}, like.device());
    const Here here(like);
    const int64_t M = integer(a[4]), N = integer(a[5]), K = integer(a[6]);
    const Operands o(a, a[14], M, 1, N, K);
    int bias_type;
    void *bias = bias_of(a[7], 0, N, &bias_type);
    Matrix res;
    if (a[9] != Py_None) res = matrix_of(matrix(a[9], "residual"), "residual", M, N);
    at::Tensor y, z;
    int y_type = MX_TYPE_BF16;
    if (a[15] != Py_None) {
        y = tensor(a[15], "out");
        const Matrix m = matrix_of(y, "out", M, N);
        if (m.pitch != N) refuse("out must be contiguous");
        y_type = m.type;
    } else if (truth(a[11])) {
        y = empty(like, {M, N}, out_type(a[10]));
        y_type = type_of(y, "y");
    }
    if (truth(a[12])) z = empty(like, {M, N}, at::kBFloat16);
    const EncodedRows e(like, a[13], M, N);
    check(mx_gemm_bias_act(o.aq, o.as, o.bq, o.bs, o.format, M, N, K, bias, bias_type, static_cast<int>(integer(a[8])), res.p,
                           res.type, res.pitch, y.defined() ? y.data_ptr() : nullptr, y_type,
                           z.defined() ? z.data_ptr() : nullptr, e.format, e.codes_p, e.scales_p, here.stream),
          "mx_gemm_bias_act");
    return tuple_of(y, z, e.codes, e.scales);
}

// bias_act_backward(dy, z, act, want_dz, want_dbias, fmt, ws) -> (dz, codes, scales, dbias)
PyObject *bias_act_backward(PyObject *const *a) {
    const at::Tensor &dy = matrix(a[0], "dy");
    on_device(a, {{1, "z"}, {6, "workspace"}}, dy.device());
    const Here here(dy);
    const int64_t T = dy.size(0), N = dy.size(1);
    const Matrix dm = matrix_of(dy, "dy", T, N);
    const int act = static_cast<int>(integer(a[2]));
    Matrix zm;
    if (a[1] != Py_None) zm = matrix_of(matrix(a[1], "z"), "z", T, N);
    else if (act != MX_ACT_NONE) refuse("an activation's gradient needs z");
    at::Tensor dz, dbias, ws;
    size_t bytes = 0;
    if (truth(a[3])) dz = empty(dy, {T, N}, at::kBFloat16);
    const EncodedRows e(dy, a[5], T, N);
    if (truth(a[4])) {
        dbias = empty(dy, {N}, at::kFloat);
        const size_t need = mx_bias_act_backward_workspace_bytes(T, N);
        if (need > 0 || a[6] != Py_None) {
            const Workspace given(dy, a[6], need);
            ws = given.t;
            bytes = given.bytes;
        }
    }
    check(mx_bias_act_backward(dm.p, dm.type, dm.pitch, zm.p, zm.type, zm.pitch, act, T, N,
                               dz.defined() ? dz.data_ptr() : nullptr, e.format, e.codes_p, e.scales_p,
                               dbias.defined() ? static_cast<float *>(dbias.data_ptr()) : nullptr,
                               ws.defined() ? ws.data_ptr() : nullptr, bytes, here.stream),
          "mx_bias_act_backward");
    return tuple_of(dz, e.codes, e.scales, dbias);
}

// expert_plan(experts, count, ws) -> (offsets, counts, slot, source)
PyObject *expert_plan(PyObject *const *a) {
    const at::Tensor &x = matrix(a[0], "experts");
    on_device(a, {{2, "workspace"}}, x.device());
    const Here here(x);
    if ((x.scalar_type() != at::kInt && x.scalar_type() != at::kLong) || !x.is_contiguous())
        refuse("experts must be contiguous and int32 or int64");
    const int64_t T = x.size(0), picks = x.size(1), count = integer(a[1]);
    if (count < 1) refuse("there must be an expert");
    if (count > MX_EXPERTS_MAX) check(MX_ERR_UNSUPPORTED, "mx_expert_plan");  // before anything is allocated for them
    // One allocation: a call for a few tokens took 7.8 us with four, 4.4 us with one.
    const Parts<4> plan(x, at::kInt, {{{count + 1}, {count}, {T, picks}, {mx_expert_rows(T, picks, count)}}});
    const at::Tensor &offsets = plan.t[0], &counts = plan.t[1], &slot = plan.t[2], &source = plan.t[3];
    at::Tensor ws;
    size_t bytes = 0;
    const size_t need = mx_expert_plan_workspace_bytes(T, picks, count);
    if (need > 0 || a[2] != Py_None) {
        const Workspace given(x, a[2], need);
        ws = given.t;
        bytes = given.bytes;
    }
    check(mx_expert_plan(x.data_ptr(), static_cast<int>(x.element_size()), T, picks, count,
                         static_cast<int32_t *>(offsets.data_ptr()), static_cast<int32_t *>(counts.data_ptr()),
                         static_cast<int32_t *>(slot.data_ptr()), static_cast<int32_t *>(source.data_ptr()),
                         ws.defined() ? ws.data_ptr() : nullptr, bytes, here.stream),
          "mx_expert_plan");
    return tuple_of(offsets, counts, slot, source);
}

// expert_dispatch(x, offsets, counts, slot, source, fmt, want_y) -> (y, codes, scales)
PyObject *expert_dispatch(PyObject *const *a) {
    const at::Tensor &x = matrix(a[0], "x");
    on_device(a, {{1, "plan.offsets"}, {2, "plan.counts"}, {3, "plan.slot"}, {4, "plan.source"}}, x.device());
    const Here here(x);
    const Plan plan(a + 1);
    const int64_t K = x.size(1);
    const Matrix m = matrix_of(x, "x", plan.T, K);
    at::Tensor y;
    if (truth(a[6])) y = empty(x, {plan.rows, K}, at::kBFloat16);
    const EncodedRows e(x, a[5], plan.rows, K);
    check(mx_expert_dispatch(m.p, m.type, m.pitch, plan.slot, plan.source, plan.T, plan.picks, plan.rows, K,
                             y.defined() ? y.data_ptr() : nullptr, e.format, e.codes_p, e.scales_p, here.stream),
          "mx_expert_dispatch");
    return tuple_of(y, e.codes, e.scales);
}

const float *weights_of(PyObject *o, const Plan &plan) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "weights");
    if (t.scalar_type() != at::kFloat || !t.is_contiguous() || t.dim() != 2 || t.size(0) != plan.T || t.size(1) != plan.picks)
        refuse("weights must be contiguous, float32 and [tokens, choices]");
    return static_cast<const float *>(t.data_ptr());
}

// expert_combine(rows, offsets, counts, slot, source, weights, residual, f32, out) -> y
PyObject *expert_combine(PyObject *const *a) {
    const at::Tensor &rows = matrix(a[0], "rows");
    on_device(a,
              {{1, "plan.offsets"}, {2, "plan.counts"}, {3, "plan.slot"}, {4, "plan.source"}, {5, "weights"}, {6, "residual"}, {8, "out"}},
              rows.device());
    const Here here(rows);
    const Plan plan(a + 1);
    const int64_t K = rows.size(1);
    const Matrix rm = matrix_of(rows, "rows", plan.rows, K);
    const float *weights = weights_of(a[5], plan);
    Matrix res;
    at::ScalarType type = rows.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
    if (a[6] != Py_None) {
        const at::Tensor &r = matrix(a[6], "residual");
        res = matrix_of(r, "residual", plan.T, K);
        type = res.type == MX_TYPE_F32 ? at::kFloat : at::kBFloat16;
    }
    if (a[7] != Py_None) type = out_type(a[7]);
    const at::Tensor y = a[8] != Py_None ? tensor(a[8], "out") : empty(rows, {plan.T, K}, type);
    const Matrix ym = matrix_of(y, "out", plan.T, K);
    if (ym.pitch != K) refuse("out must be contiguous");
    check(mx_expert_combine(rm.p, rm.type, rm.pitch, plan.slot, weights, plan.T, plan.picks, plan.rows, K, res.p, res.type,
                            res.pitch, ym.p, ym.type, here.stream),
          "mx_expert_combine");
    return wrap(y);
}

// expert_combine_backward(dy, rows, offsets, counts, slot, source, weights, fmt, want_y, want_dweights)
//   -> (drows, codes, scales, dweights)
PyObject *expert_combine_backward(PyObject *const *a) {
    const at::Tensor &dy = matrix(a[0], "dy");
    on_device(a, {{1, "rows"}, {2, "plan.offsets"}, {3, "plan.counts"}, {4, "plan.slot"}, {5, "plan.source"}, {6, "weights"}},
              dy.device());
    const Here here(dy);
    const Plan plan(a + 2);
    const int64_t K = dy.size(1);
    const Matrix dm = matrix_of(dy, "dy", plan.T, K);
    const float *weights = weights_of(a[6], plan);
    Matrix rm;
    at::Tensor drows, dweights;
    if (truth(a[9])) {
        if (a[1] == Py_None) refuse("dweights need rows");
        rm = matrix_of(matrix(a[1], "rows"), "rows", plan.rows, K);
        dweights = empty(dy, {plan.T, plan.picks}, at::kFloat);
    }
    if (a[6] == Py_None) refuse("weights must be a torch.Tensor");  // no tokens: a tensor without memory
    if (truth(a[8])) drows = empty(dy, {plan.rows, K}, at::kBFloat16);
    const EncodedRows e(dy, a[7], plan.rows, K);
    check(mx_expert_combine_backward(dm.p, dm.type, dm.pitch, rm.p, rm.type, rm.pitch, plan.slot, plan.source, weights, plan.T,
                                     plan.picks, plan.rows, K, drows.defined() ? drows.data_ptr() : nullptr, e.format,
                                     e.codes_p, e.scales_p,
                                     dweights.defined() ? static_cast<float *>(dweights.data_ptr()) : nullptr, here.stream),
          "mx_expert_combine_backward");
    return tuple_of(drows, e.codes, e.scales, dweights);
}

// quantize_experts(w, contract, operands, rot, rot_block, seed) -> (codes, scales)
PyObject *quantize_experts(PyObject *const *a) {
    const at::Tensor &w = tensor(a[0], "w");
    if (w.dim() != 3 || !w.is_contiguous()) refuse("w must be contiguous and [experts, rows, columns]");
    if (type_of(w, "w") != MX_TYPE_BF16) refuse("w must be bf16 (torch.bfloat16 or raw 16-bit patterns)");
    const Here here(w);
    const int64_t E = w.size(0), rows = w.size(1), cols = w.size(2), contract = integer(a[1]);
    const int operands = operands_of(a[2]);
    const int64_t lines = contract == MX_CONTRACT_ROWS ? cols : rows, k = contract == MX_CONTRACT_ROWS ? rows : cols;
    const int64_t row_bytes = operands == MX_FORMAT_MXFP8 ? k : k / 2;
    const at::Tensor codes = empty(w, {E * lines, row_bytes}, at::kByte),
                     scales = empty(w, {std::max<int64_t>(1, E * static_cast<int64_t>(mx_scales_bytes(lines, k)))}, at::kByte);
    check(mx_quantize_experts(w.data_ptr(), E, rows, cols, operands, static_cast<int>(contract), static_cast<int>(integer(a[3])),
                              static_cast<int>(integer(a[4])), bits(a[5]), codes.data_ptr(),
                              scales.data_ptr(), here.stream),
          "mx_quantize_experts");
    return tuple_of(codes, scales);
}

// gemm_experts(Aq, As, Bq, Bs, offsets, counts, slot, source, N, K, bias, act, f32, want_y, want_z, fmt, operands)
//   -> (y, z, codes, scales)
PyObject *gemm_experts(PyObject *const *a) {
    const at::Tensor &like = tensor(a[0], "Aq");
    on_device(a,
              {{1, "As"}, {2, "Bq"}, {3, "Bs"}, {4, "plan.offsets"}, {5, "plan.counts"}, {6, "plan.slot"}, {7, "plan.source"}, {10, "bias"}},
              like.device());
    const Here here(like);
    const Plan plan(a + 4);
    const int64_t N = integer(a[8]), K = integer(a[9]);
    const Operands o(a, a[16], plan.rows, plan.experts, N, K);
    int bias_type;
    void *bias = bias_of(a[10], plan.experts, N, &bias_type);
    at::Tensor y, z;
    const at::ScalarType type = out_type(a[12]);
    if (truth(a[13])) y = empty(like, {plan.rows, N}, type);
    if (truth(a[14])) z = empty(like, {plan.rows, N}, at::kBFloat16);
    const EncodedRows e(like, a[15], plan.rows, N);
    check(mx_gemm_experts(o.aq, o.as, o.bq, o.bs, o.format, plan.offsets, plan.counts, plan.experts, plan.rows, N, K, bias,
                          bias_type, static_cast<int>(integer(a[11])), y.defined() ? y.data_ptr() : nullptr,
                          type == at::kFloat ? MX_TYPE_F32 : MX_TYPE_BF16, z.defined() ? z.data_ptr() : nullptr, e.format,
                          e.codes_p, e.scales_p, here.stream),
          "mx_gemm_experts");
    return tuple_of(y, z, e.codes, e.scales);
}

// An output [experts, M, N] of either type: the one given, or a new one.
at::Tensor stack_of(PyObject *given, const at::Tensor &like, at::ScalarType type, int64_t E, int64_t M, int64_t N) {
    if (given == Py_None) return empty(like, {E, M, N}, type);
    const at::Tensor &t = tensor(given, "out");
    if (t.dim() != 3 || t.size(0) != E || t.size(1) != M || t.size(2) != N || !t.is_contiguous())
        refuse("out must be contiguous and [%lld, %lld, %lld]", static_cast<long long>(E), static_cast<long long>(M),
               static_cast<long long>(N));
    return t;
}

// gemm_experts_wgrad(Aq, As, Bq, Bs, offsets, counts, slot, source, M, N, f32, operands, out) -> C
PyObject *gemm_experts_wgrad(PyObject *const *a) {
    const at::Tensor &like = tensor(a[0], "Aq");
    on_device(a,
              {{1, "As"}, {2, "Bq"}, {3, "Bs"}, {4, "plan.offsets"}, {5, "plan.counts"}, {6, "plan.slot"}, {7, "plan.source"}, {12, "out"}},
              like.device());
    const Here here(like);
    const Plan plan(a + 4);
    const int64_t M = integer(a[8]), N = integer(a[9]);
    const Operands o(a, a[11], M, 1, N, plan.rows);
    const at::Tensor c = stack_of(a[12], like, out_type(a[10]), plan.experts, M, N);
    check(mx_gemm_experts_wgrad(o.aq, o.as, o.bq, o.bs, o.format, plan.offsets, plan.experts, plan.rows, M, N, c.data_ptr(),
                                type_of(c, "out"), here.stream),
          "mx_gemm_experts_wgrad");
    return wrap(c);
}

// linear_experts_wgrad(dY, X, offsets, counts, slot, source, operands, rot, rot_block, rnd, seed, f32, ws, out) -> dW
PyObject *linear_experts_wgrad(PyObject *const *a) {
    const at::Tensor &dY = matrix(a[0], "dY"), &X = matrix(a[1], "X");
    on_device(a,
              {{1, "X"}, {2, "plan.offsets"}, {3, "plan.counts"}, {4, "plan.slot"}, {5, "plan.source"}, {12, "workspace"}, {13, "out"}},
              dY.device());
    const Here here(dY);
    const Plan plan(a + 2);
    const int64_t N = dY.size(1), K = X.size(1);
    const Matrix dm = matrix_of(dY, "dY", plan.rows, N), xm = matrix_of(X, "X", plan.rows, K);
    if (dm.type != MX_TYPE_BF16 || xm.type != MX_TYPE_BF16 || dm.pitch != N || xm.pitch != K)
        refuse("dY and X must be contiguous and bf16 (torch.bfloat16 or raw 16-bit patterns)");
    const int operands = operands_of(a[6]);
    const at::Tensor dW = stack_of(a[13], dY, out_type(a[11]), plan.experts, N, K);
    const Workspace ws(dY, a[12], mx_linear_experts_wgrad_workspace_bytes(operands, plan.rows, N, K));
    check(mx_linear_experts_wgrad(dm.p, xm.p, operands, plan.offsets, plan.experts, plan.rows, N, K,
                                  static_cast<int>(integer(a[7])), static_cast<int>(integer(a[8])),
                                  static_cast<int>(integer(a[9])), bits(a[10]), dW.data_ptr(),
                                  type_of(dW, "out"), ws.t.data_ptr(), ws.bytes, here.stream),
          "mx_linear_experts_wgrad");
    return wrap(dW);
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
                           method<gemm_bias_act, 16>("gemm_bias_act"),
                           method<bias_act_backward, 7>("bias_act_backward"),
                           method<expert_plan, 3>("expert_plan"),
                           method<expert_dispatch, 7>("expert_dispatch"),
                           method<expert_combine, 9>("expert_combine"),
                           method<expert_combine_backward, 10>("expert_combine_backward"),
                           method<quantize_experts, 6>("quantize_experts"),
                           method<gemm_experts, 17>("gemm_experts"),
                           method<gemm_experts_wgrad, 13>("gemm_experts_wgrad"),
                           method<linear_experts_wgrad, 14>("linear_experts_wgrad"),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mx_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mx_torch() { return PyModule_Create(&g_module); }
