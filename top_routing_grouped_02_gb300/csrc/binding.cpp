// Python entry points of the sub-block calls (layer norm, residual dropout, dense
// feed-forward block): argument checks, output allocation and one call into
// libmoe.so each. They do what the ctypes functions of moe.py do for the other calls;
// these run at sizes where a call's host time is several times its GPU time, and from
// Python it was (12 us of host time for a 2 us kernel).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>

#include "moe.h"

namespace {

PyObject *g_error = nullptr;  // moe.MoeError

using Refused = python_error;  // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const char *format, const char *name) {
    PyErr_Format(type, format, name);
    throw Refused();
}

at::Tensor tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}
at::Tensor optional_tensor(PyObject *o, const char *name) {
    return o == Py_None ? at::Tensor() : tensor(o, name);
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
long integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
uint64_t word(PyObject *o) {
    const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
    if (v == (uint64_t)-1 && PyErr_Occurred()) throw Refused();
    return v;
}

int type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return MOE_DTYPE_BF16;
        case at::kHalf: return MOE_DTYPE_F16;
        case at::kFloat: return MOE_DTYPE_F32;
        default: return -1;
    }
}

// Every operand and the given stream belong to the first tensor's device.
struct Named {
    const at::Tensor &t;
    const char *name;
};
void one_device(const Named &first, std::initializer_list<Named> others, PyObject *stream) {
    if (!first.t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", first.name);
    const int device = first.t.get_device();
    for (const Named &o : others)
        if (o.t.defined() && (!o.t.is_cuda() || o.t.get_device() != device))
            refuse(PyExc_ValueError, "%s must lie on the first tensor's device", o.name);
    if (stream == Py_None) return;
    PyObject *v = PyObject_GetAttrString(stream, "device_index");
    if (v == nullptr) {  // a bare handle: the caller's word for it
        PyErr_Clear();
        return;
    }
    const long index = PyLong_AsLong(v);
    Py_DECREF(v);
    if (index == -1 && PyErr_Occurred()) throw Refused();
    if (index != device) refuse(PyExc_ValueError, "%s must belong to the first tensor's device", "stream");
}

// The call's device and stream, torch's current ones while the call lasts: its kernels are
// launched on that device, and what it allocates (outputs, scratch) comes from that
// stream's memory, which no pending work of another stream still uses or will be given
// before the call's kernels are done.
struct OnStream {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    cudaStream_t s;
    OnStream(PyObject *o, const at::Tensor &t) : device(t.device()) {
        s = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
        if (o == Py_None) return;
        PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
        if (v == nullptr) throw Refused();
        const uint64_t h = PyLong_AsUnsignedLongLongMask(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw Refused();
        if (reinterpret_cast<cudaStream_t>(h) == s) return;
        s = reinterpret_cast<cudaStream_t>(h);
        guard.emplace(c10::cuda::getStreamFromExternal(s, t.get_device()));
    }
    operator void *() const { return s; }
};

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// A tensor seen as a matrix of rows along its last dimension: contiguous, or 2-D with
// unit inner stride.
struct Rows {
    void *p;
    int64_t ld, T, d;
};
Rows rows_of(const at::Tensor &t, const char *name, const at::Tensor *like = nullptr) {
    if (!t.is_cuda() || type_of(t) < 0 || t.dim() < 1)
        refuse(PyExc_ValueError, "%s must be a bf16, fp16 or fp32 CUDA tensor", name);
    if (like != nullptr && (t.sizes() != like->sizes() || t.scalar_type() != like->scalar_type() ||
                            t.get_device() != like->get_device()))
        refuse(PyExc_ValueError, "%s must have the first tensor's shape, type and device", name);
    Rows r;
    r.p = t.data_ptr();
    r.d = t.size(-1);
    if (r.d == 0 || r.d > INT32_MAX) refuse(PyExc_ValueError, "%s has rows of an unsupported length", name);
    if (t.is_contiguous()) {
        r.ld = r.d;
        r.T = t.numel() / r.d;
        return r;
    }
    if (t.dim() != 2 || (r.d > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < r.d))
        refuse(PyExc_ValueError, "%s must be contiguous or a matrix of non-overlapping rows", name);
    r.ld = t.stride(0);
    r.T = t.size(0);
    return r;
}
// An output: `given`, or a new contiguous tensor like x.
at::Tensor output(const at::Tensor &given, const at::Tensor &x) {
    return given.defined() ? given : fresh(x.sizes(), x.scalar_type(), x);
}
void *vec_of(const at::Tensor &t, int64_t d, const at::Tensor &x, const char *name) {
    if (!t.defined()) return nullptr;
    if (!t.is_cuda() || t.dim() != 1 || t.size(0) != d || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous CUDA vector of the rows' length", name);
    if (t.scalar_type() != x.scalar_type() && t.scalar_type() != at::kFloat)
        refuse(PyExc_TypeError, "%s must have the rows' type or be fp32", name);
    return t.data_ptr();
}
float *stat_of(const at::Tensor &t, int64_t T, const char *name) {
    if (!t.is_cuda() || t.scalar_type() != at::kFloat || !t.is_contiguous() || t.numel() != T)
        refuse(PyExc_ValueError, "%s must hold one contiguous fp32 value a row", name);
    return static_cast<float *>(t.data_ptr());
}
const uint64_t *counter_of(const at::Tensor &t) {
    if (!t.defined()) return nullptr;
    if (!t.is_cuda() || t.scalar_type() != at::kLong || t.numel() != 1)
        refuse(PyExc_ValueError, "%s must be a one-element int64 CUDA tensor", "offset_dev");
    return static_cast<const uint64_t *>(t.data_ptr());
}
void *dense(const at::Tensor &t, at::IntArrayRef sizes, at::ScalarType type, const char *name) {
    if (!t.is_cuda() || !t.is_contiguous() || t.scalar_type() != type || t.sizes() != sizes)
        refuse(PyExc_ValueError, "%s must be a contiguous CUDA tensor of the call's shape and type", name);
    return t.data_ptr();
}
moe_dtype_t dtype(const at::Tensor &t) { return static_cast<moe_dtype_t>(type_of(t)); }

void check(const char *fn, moe_status_t status) {
    if (status == MOE_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "si", fn, (int)status);
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}

void expect(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw Refused();
}
PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <typename... Ts>
PyObject *wrap_all(const Ts &...ts) {
    PyObject *items[] = {wrap(ts)...};
    PyObject *tuple = PyTuple_New(sizeof...(ts));
    for (size_t i = 0; i < sizeof...(ts); ++i) PyTuple_SET_ITEM(tuple, i, items[i]);
    return tuple;
}

// x, gamma, beta, eps, stats, y, stream
PyObject *layernorm(PyObject *const *a, Py_ssize_t n) {
    expect(n, 7);
    const at::Tensor x = tensor(a[0], "x");
    const at::Tensor gamma = optional_tensor(a[1], "gamma"), beta = optional_tensor(a[2], "beta"),
                     given = optional_tensor(a[5], "y");
    one_device({x, "x"}, {{gamma, "gamma"}, {beta, "beta"}, {given, "y"}}, a[6]);
    const Rows rx = rows_of(x, "x");
    const OnStream stream(a[6], x);
    const double eps = number(a[3]);
    const bool stats = truth(a[4]);
    void *pg = vec_of(gamma, rx.d, x, "gamma"), *pb = vec_of(beta, rx.d, x, "beta");
    if (pg != nullptr && pb != nullptr && gamma.scalar_type() != beta.scalar_type())
        refuse(PyExc_TypeError, "gamma and %s must have one type", "beta");
    const at::Tensor y = output(given, x);
    const Rows ry = rows_of(y, "y", &x);
    at::Tensor mean, rstd;
    if (stats) {
        const auto sizes = x.sizes().slice(0, x.dim() - 1);
        mean = fresh(sizes, at::kFloat, x);
        rstd = fresh(sizes, at::kFloat, x);
    }
    check("moe_layernorm_forward",
          moe_layernorm_forward(rx.p, rx.ld, pg, pb, rx.T, (int)rx.d, (float)eps, dtype(x),
                                dtype(pg != nullptr ? gamma : pb != nullptr ? beta : x), ry.p, ry.ld,
                                stats ? static_cast<float *>(mean.data_ptr()) : nullptr,
                                stats ? static_cast<float *>(rstd.data_ptr()) : nullptr,
                                stream));
    return stats ? wrap_all(y, mean, rstd) : wrap(y);
}

// dy, x, gamma, mean, rstd, dres, fp32 weight gradients without gamma, dx, scratch, stream
PyObject *layernorm_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 10);
    const at::Tensor dy = tensor(a[0], "dy"), x = tensor(a[1], "x");
    const at::Tensor gamma = optional_tensor(a[2], "gamma"), mean = tensor(a[3], "mean"),
                     rstd = tensor(a[4], "rstd"), dres = optional_tensor(a[5], "dres"),
                     given = optional_tensor(a[7], "dx"), memory = optional_tensor(a[8], "scratch");
    one_device({x, "x"},
               {{dy, "dy"}, {gamma, "gamma"}, {mean, "mean"}, {rstd, "rstd"}, {dres, "dres"}, {given, "dx"},
                {memory, "scratch"}},
               a[9]);
    const Rows rx = rows_of(x, "x"), rdy = rows_of(dy, "dy", &x);
    const OnStream stream(a[9], x);
    Rows rr{};
    if (dres.defined()) rr = rows_of(dres, "dres", &x);
    void *pg = vec_of(gamma, rx.d, x, "gamma");
    float *pm = stat_of(mean, rx.T, "mean"), *pr = stat_of(rstd, rx.T, "rstd");
    const at::Tensor dx = output(given, x);
    const Rows rdx = rows_of(dx, "dx", &x);
    const at::ScalarType wt = gamma.defined()               ? gamma.scalar_type()
                              : truth(a[6]) ? at::kFloat
                                                            : x.scalar_type();
    const at::Tensor dgamma = fresh({rx.d}, wt, x);
    const at::Tensor dbeta = fresh({rx.d}, wt, x);
    const at::Tensor scratch =
        memory.defined() ? memory
                         : fresh({(int64_t)moe_layernorm_scratch_bytes(rx.T, (int)rx.d)}, at::kByte, x);
    if (!scratch.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "scratch");
    check("moe_layernorm_backward",
          moe_layernorm_backward(rdy.p, rdy.ld, rx.p, rx.ld, pg, pm, pr, rr.p, rr.ld, rx.T, (int)rx.d,
                                 dtype(x), dtype(dgamma), rdx.p, rdx.ld, dgamma.data_ptr(),
                                 dbeta.data_ptr(), scratch.data_ptr(), scratch.nbytes(),
                                 stream));
    return wrap_all(dx, dgamma, dbeta);
}

// x, p, seed, offset, residual, offset_dev, y, stream
PyObject *dropout(PyObject *const *a, Py_ssize_t n) {
    expect(n, 8);
    const at::Tensor x = tensor(a[0], "x"), res = optional_tensor(a[4], "residual"),
                     ctr = optional_tensor(a[5], "offset_dev"), given = optional_tensor(a[6], "y");
    one_device({x, "x"}, {{res, "residual"}, {ctr, "offset_dev"}, {given, "y"}}, a[7]);
    const Rows rx = rows_of(x, "x");
    const OnStream stream(a[7], x);
    const double p = number(a[1]);
    const uint64_t seed = word(a[2]), offset = word(a[3]);
    Rows rr{};
    if (res.defined()) rr = rows_of(res, "residual", &x);
    const uint64_t *pc = counter_of(ctr);
    const at::Tensor y = output(given, x);
    const Rows ry = rows_of(y, "y", &x);
    check("moe_dropout", moe_dropout(rx.p, rx.ld, rr.p, rr.ld, rx.T, (int)rx.d, p, seed, offset, pc,
                                     dtype(x), ry.p, ry.ld, stream));
    return wrap(y);
}

// dy, p, seed, offset, offset_dev, dx, stream
PyObject *dropout_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 7);
    const at::Tensor dy = tensor(a[0], "dy"), ctr = optional_tensor(a[4], "offset_dev"),
                     given = optional_tensor(a[5], "dx");
    one_device({dy, "dy"}, {{ctr, "offset_dev"}, {given, "dx"}}, a[6]);
    const Rows r = rows_of(dy, "dy");
    const OnStream stream(a[6], dy);
    const double p = number(a[1]);
    const uint64_t seed = word(a[2]), offset = word(a[3]);
    const uint64_t *pc = counter_of(ctr);
    const at::Tensor dx = output(given, dy);
    const Rows rdx = rows_of(dx, "dx", &dy);
    check("moe_dropout_backward",
          moe_dropout_backward(r.p, r.ld, r.T, (int)r.d, p, seed, offset, pc, dtype(dy), rdx.p, rdx.ld,
                               stream));
    return wrap(dx);
}

// The feed-forward block's operands.
struct Ffn {
    at::Tensor x, W1, W3, W2, ws;
    int T, d, n;
    void *px, *p1, *p3, *p2, *pws;
    at::ScalarType type;
};
Ffn ffn_args(PyObject *x, PyObject *W1, PyObject *W3, PyObject *W2, PyObject *ws, PyObject *stream) {
    Ffn f{tensor(x, "x"), tensor(W1, "W1"), tensor(W3, "W3"), tensor(W2, "W2"), tensor(ws, "ws")};
    one_device({f.x, "x"}, {{f.W1, "W1"}, {f.W3, "W3"}, {f.W2, "W2"}, {f.ws, "ws"}}, stream);
    if (f.x.dim() < 1 || f.W1.dim() != 2 || f.x.size(-1) != f.W1.size(0))
        refuse(PyExc_ValueError, "%s must be [..., d] and W1 [d, n]", "x");
    f.type = f.x.scalar_type();
    if (f.type != at::kBFloat16 && f.type != at::kHalf)
        refuse(PyExc_TypeError, "the feed-forward block takes bf16 or fp16 %s", "x");
    const int64_t d = f.W1.size(0), n = f.W1.size(1), T = d > 0 ? f.x.numel() / d : 0;
    if (T > INT32_MAX || d > INT32_MAX || n > INT32_MAX)
        refuse(PyExc_ValueError, "%s is too large", "x");
    f.px = dense(f.x, f.x.sizes(), f.type, "x");
    f.p1 = dense(f.W1, {d, n}, f.type, "W1");
    f.p3 = dense(f.W3, {d, n}, f.type, "W3");
    f.p2 = dense(f.W2, {n, d}, f.type, "W2");
    if (!f.ws.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "ws");
    f.pws = f.ws.data_ptr();
    f.T = (int)T;
    f.d = (int)d;
    f.n = (int)n;
    return f;
}

// x, W1, W3, W2, act, ws, Y, stream
PyObject *ffn(PyObject *const *a, Py_ssize_t n) {
    expect(n, 8);
    const Ffn f = ffn_args(a[0], a[1], a[2], a[3], a[5], a[7]);
    const at::Tensor given = optional_tensor(a[6], "Y");
    one_device({f.x, "x"}, {{given, "Y"}}, Py_None);
    const OnStream stream(a[7], f.x);
    const at::Tensor Y = output(given, f.x);
    void *py = dense(Y, f.x.sizes(), f.type, "Y");
    check("moe_ffn_forward",
          moe_ffn_forward(f.px, f.p1, f.p3, f.p2, f.T, f.d, f.n, (moe_act_t)integer(a[4]), dtype(f.x), py,
                          f.pws, f.ws.nbytes(), stream));
    return wrap(Y);
}

// x, W1, W3, W2, act, ws, stream
PyObject *ffn_train(PyObject *const *a, Py_ssize_t n) {
    expect(n, 7);
    const Ffn f = ffn_args(a[0], a[1], a[2], a[3], a[5], a[6]);
    const OnStream stream(a[6], f.x);
    const at::Tensor Y = fresh(f.x.sizes(), f.type, f.x);
    const at::Tensor H = fresh({f.T, f.n}, f.type, f.x);
    const int64_t saved = (int64_t)moe_ffn_saved_floats(f.T, f.n);
    const at::Tensor F1 = fresh({saved}, at::kFloat, f.x);
    const at::Tensor F3 = fresh({saved}, at::kFloat, f.x);
    check("moe_ffn_forward_train",
          moe_ffn_forward_train(f.px, f.p1, f.p3, f.p2, f.T, f.d, f.n, (moe_act_t)integer(a[4]),
                                dtype(f.x), Y.data_ptr(), H.data_ptr(),
                                static_cast<float *>(F1.data_ptr()), static_cast<float *>(F3.data_ptr()),
                                f.pws, f.ws.nbytes(), stream));
    return wrap_all(Y, H, F1, F3);
}

// dY, x, W1, W3, W2, H, F1, F3, act, need_dx, need_dw, ws, stream
PyObject *ffn_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 13);
    const Ffn f = ffn_args(a[1], a[2], a[3], a[4], a[11], a[12]);
    const at::Tensor dY = tensor(a[0], "dY"), H = tensor(a[5], "H"), F1 = tensor(a[6], "F1"),
                     F3 = tensor(a[7], "F3");
    one_device({f.x, "x"}, {{dY, "dY"}, {H, "H"}, {F1, "F1"}, {F3, "F3"}}, Py_None);
    const OnStream stream(a[12], f.x);
    const int64_t saved = (int64_t)moe_ffn_saved_floats(f.T, f.n);
    void *pdy = dense(dY, f.x.sizes(), f.type, "dY"), *ph = dense(H, {f.T, f.n}, f.type, "H");
    const float *pf1 = static_cast<float *>(dense(F1, {saved}, at::kFloat, "F1"));
    const float *pf3 = static_cast<float *>(dense(F3, {saved}, at::kFloat, "F3"));
    at::Tensor dX, dW1, dW3, dW2;
    if (truth(a[9])) dX = fresh(f.x.sizes(), f.type, f.x);
    const bool dw = truth(a[10]);
    if (dw) {
        dW1 = fresh({f.d, f.n}, f.type, f.x);
        dW3 = fresh({f.d, f.n}, f.type, f.x);
        dW2 = fresh({f.n, f.d}, f.type, f.x);
    }
    check("moe_ffn_backward",
          moe_ffn_backward(pdy, f.px, f.p1, f.p3, f.p2, ph, pf1, pf3, f.T, f.d, f.n,
                           (moe_act_t)integer(a[8]), dtype(f.x), dX.defined() ? dX.data_ptr() : nullptr,
                           dw ? dW1.data_ptr() : nullptr, dw ? dW3.data_ptr() : nullptr,
                           dw ? dW2.data_ptr() : nullptr, f.pws, f.ws.nbytes(), stream));
    return wrap_all(dX, dW1, dW3, dW2);
}

// error class
PyObject *set_error(PyObject *const *a, Py_ssize_t n) {
    expect(n, 1);
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

// No C++ exception leaves an entry point: torch's macros translate them (a refusal's Python
// exception is set already) and give torch's pending warnings first.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return F(args, n);
    END_HANDLE_TH_ERRORS
}

#define MOE_ENTRY(F) {#F, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MOE_ENTRY(layernorm), MOE_ENTRY(layernorm_backward), MOE_ENTRY(dropout),
                           MOE_ENTRY(dropout_backward), MOE_ENTRY(ffn), MOE_ENTRY(ffn_train),
                           MOE_ENTRY(ffn_backward), MOE_ENTRY(set_error),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
