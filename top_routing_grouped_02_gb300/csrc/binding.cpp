// Python entry points of the sub-block calls (layer norm, residual dropout, dense feed-forward
// block, projections, norms around a block, dispatch and combine): argument checks, output allocation and one call into
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
#include <vector>

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

// A block's gate: a matrix like x, or one fp32 value a row.
struct Gate {
    moe_gate_t kind = MOE_GATE_NONE;
    void *p = nullptr;
    int64_t ld = 0;
};
Gate gate_of(const at::Tensor &t, const at::Tensor &x, const Rows &rx, const char *name) {
    Gate g;
    if (!t.defined()) return g;
    if (t.dim() == x.dim()) {
        const Rows r = rows_of(t, name, &x);
        g.kind = MOE_GATE_FULL;
        g.p = r.p;
        g.ld = r.ld;
        return g;
    }
    if (t.sizes() != x.sizes().slice(0, x.dim() - 1))
        refuse(PyExc_ValueError, "%s must have x's shape, or that of its rows", name);
    g.kind = MOE_GATE_ROW;
    g.p = stat_of(t, rx.T, name);
    return g;
}
Rows rows_if(const at::Tensor &t, const char *name, const at::Tensor &like) {
    return t.defined() ? rows_of(t, name, &like) : Rows{};
}
moe_dtype_t weight_type(const at::Tensor &post, const at::Tensor &pre, const at::Tensor &x) {
    if (post.defined() && pre.defined() && post.scalar_type() != pre.scalar_type())
        refuse(PyExc_TypeError, "post and %s must have one type", "pre");
    return dtype(post.defined() ? post : pre.defined() ? pre : x);
}
int norms_of(bool post, bool pre) { return (post ? MOE_NORM_POST : 0) | (pre ? MOE_NORM_PRE : 0); }

// x, b, post, pre, gate, scale, eps, post_norm, pre_norm, stats, y, u, stream
PyObject *block_norm(PyObject *const *a, Py_ssize_t n) {
    expect(n, 13);
    const at::Tensor x = tensor(a[0], "x"), b = optional_tensor(a[1], "b"), post = optional_tensor(a[2], "post"),
                     pre = optional_tensor(a[3], "pre"), gate = optional_tensor(a[4], "gate"),
                     given_y = optional_tensor(a[10], "y"), given_u = optional_tensor(a[11], "u");
    one_device({x, "x"},
               {{b, "b"}, {post, "post"}, {pre, "pre"}, {gate, "gate"}, {given_y, "y"}, {given_u, "u"}}, a[12]);
    const Rows rx = rows_of(x, "x"), rb = rows_if(b, "b", x);
    const OnStream stream(a[12], x);
    const double scale = number(a[5]), eps = number(a[6]);
    const bool post_norm = truth(a[7]), pre_norm = truth(a[8]), stats = truth(a[9]);
    void *pp = vec_of(post, rx.d, x, "post"), *pq = vec_of(pre, rx.d, x, "pre");
    const moe_dtype_t wt = weight_type(post, pre, x);
    const Gate g = gate_of(gate, x, rx, "gate");
    at::Tensor y, u, r_post, r_pre;
    if (b.defined()) y = output(given_y, x);
    else if (given_y.defined()) refuse(PyExc_ValueError, "without a block there is no %s", "y");
    if (pre_norm) u = output(given_u, x);
    else if (given_u.defined()) refuse(PyExc_ValueError, "without the pre norm there is no %s", "u");
    const Rows ry = rows_if(y, "y", x), ru = rows_if(u, "u", x);
    const auto sizes = x.sizes().slice(0, x.dim() - 1);
    if (stats && post_norm) r_post = fresh(sizes, at::kFloat, x);
    if (stats && pre_norm) r_pre = fresh(sizes, at::kFloat, x);
    auto floats = [](const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; };
    check("moe_block_norm_forward",
          moe_block_norm_forward(rx.p, rx.ld, rb.p, rb.ld, g.p, g.ld, g.kind, pp, pq, (float)scale,
                                 norms_of(post_norm, pre_norm), rx.T, (int)rx.d, (float)eps, dtype(x), wt, ry.p,
                                 ry.ld, ru.p, ru.ld, floats(r_post), floats(r_pre), stream));
    return stats ? wrap_all(y, u, r_post, r_pre) : wrap_all(y, u);
}

// dy, du, x, b, post, pre, rstd_post, rstd_pre, gate, scale, fp32 weight gradients without
// weights, dx, db, scratch, stream
PyObject *block_norm_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 15);
    const at::Tensor dy = optional_tensor(a[0], "dy"), du = optional_tensor(a[1], "du"), x = tensor(a[2], "x"),
                     b = optional_tensor(a[3], "b"), post = optional_tensor(a[4], "post"),
                     pre = optional_tensor(a[5], "pre"), r_post = optional_tensor(a[6], "rstd_post"),
                     r_pre = optional_tensor(a[7], "rstd_pre"), gate = optional_tensor(a[8], "gate"),
                     given_dx = optional_tensor(a[11], "dx"), given_db = optional_tensor(a[12], "db"),
                     memory = optional_tensor(a[13], "scratch");
    one_device({x, "x"},
               {{dy, "dy"}, {du, "du"}, {b, "b"}, {post, "post"}, {pre, "pre"}, {r_post, "rstd_post"},
                {r_pre, "rstd_pre"}, {gate, "gate"}, {given_dx, "dx"}, {given_db, "db"}, {memory, "scratch"}},
               a[14]);
    const Rows rx = rows_of(x, "x"), rb = rows_if(b, "b", x), rdy = rows_if(dy, "dy", x), rdu = rows_if(du, "du", x);
    const OnStream stream(a[14], x);
    const double scale = number(a[9]);
    void *pp = vec_of(post, rx.d, x, "post"), *pq = vec_of(pre, rx.d, x, "pre");
    moe_dtype_t wt = weight_type(post, pre, x);
    if (pp == nullptr && pq == nullptr && truth(a[10])) wt = MOE_DTYPE_F32;
    const Gate g = gate_of(gate, x, rx, "gate");
    const float *pr = r_post.defined() ? stat_of(r_post, rx.T, "rstd_post") : nullptr;
    const float *qr = r_pre.defined() ? stat_of(r_pre, rx.T, "rstd_pre") : nullptr;
    const at::Tensor dx = output(given_dx, x);
    at::Tensor db, dgate, dpost, dpre;
    if (b.defined()) db = output(given_db, x);
    else if (given_db.defined()) refuse(PyExc_ValueError, "without a block there is no %s", "db");
    if (gate.defined()) dgate = fresh(gate.sizes(), gate.scalar_type(), x);
    const at::ScalarType wtype = wt == MOE_DTYPE_F32 ? at::kFloat : x.scalar_type();
    if (b.defined()) dpost = fresh({rx.d}, wtype, x);
    if (r_pre.defined()) dpre = fresh({rx.d}, wtype, x);
    const at::Tensor scratch =
        memory.defined() ? memory
                         : fresh({(int64_t)moe_block_norm_scratch_bytes(rx.T, (int)rx.d)}, at::kByte, x);
    if (!scratch.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "scratch");
    const Rows rdx = rows_of(dx, "dx", &x), rdb = rows_if(db, "db", x);
    auto data = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    check("moe_block_norm_backward",
          moe_block_norm_backward(rdy.p, rdy.ld, rdu.p, rdu.ld, rx.p, rx.ld, rb.p, rb.ld, g.p, g.ld, g.kind, pp, pq,
                                  (float)scale, norms_of(r_post.defined(), r_pre.defined()), pr, qr, rx.T,
                                  (int)rx.d, dtype(x), wt, rdx.p, rdx.ld, rdb.p, rdb.ld, data(dgate), rx.d,
                                  data(dpost), data(dpre), scratch.data_ptr(), scratch.nbytes(), stream));
    return wrap_all(dx, db, dgate, dpost, dpre);
}

// The map of slots onto sorted rows.
const int32_t *slots_of(const at::Tensor &t, int64_t slots) {
    if (!t.is_cuda() || t.scalar_type() != at::kInt || !t.is_contiguous() || t.numel() != slots)
        refuse(PyExc_ValueError, "%s must hold one contiguous int32 value a slot", "row_of_slot");
    return static_cast<const int32_t *>(t.data_ptr());
}
// Rows in another order than the first tensor's: as long and of its type.
Rows sorted_rows(const at::Tensor &t, const at::Tensor &like, int64_t d, const char *name) {
    const Rows r = rows_of(t, name);
    if (t.dim() != 2 || r.d != d || t.scalar_type() != like.scalar_type())
        refuse(PyExc_ValueError, "%s must be a matrix of rows of the call's length and type", name);
    return r;
}
int slots_a_token(int64_t K) {
    if (K < 1 || K > INT32_MAX) refuse(PyExc_ValueError, "%s must be positive", "K");
    return (int)K;
}

// x, row_of_slot, K, xg, stream
PyObject *dispatch(PyObject *const *a, Py_ssize_t n) {
    expect(n, 5);
    const at::Tensor x = tensor(a[0], "x"), map = tensor(a[1], "row_of_slot"), given = optional_tensor(a[3], "xg");
    one_device({x, "x"}, {{map, "row_of_slot"}, {given, "xg"}}, a[4]);
    const Rows rx = rows_of(x, "x");
    const int K = slots_a_token(integer(a[2]));
    const int32_t *pm = slots_of(map, rx.T * K);
    const OnStream stream(a[4], x);
    const at::Tensor xg = given.defined() ? given : fresh({rx.T * K, rx.d}, x.scalar_type(), x);
    const Rows rg = sorted_rows(xg, x, rx.d, "xg");
    check("moe_dispatch", moe_dispatch(rx.p, rx.ld, pm, rx.T, K, (int)rx.d, dtype(x), rg.p, rg.ld, rg.T, stream));
    return wrap(xg);
}

// z, row_of_slot, w or the slots a token, residual, y, stream
PyObject *combine_weighted(PyObject *const *a, Py_ssize_t n) {
    expect(n, 6);
    const at::Tensor z = tensor(a[0], "z"), map = tensor(a[1], "row_of_slot"),
                     res = optional_tensor(a[3], "residual"), given = optional_tensor(a[4], "y");
    at::Tensor w;
    int K;
    if (PyLong_Check(a[2])) {
        K = slots_a_token(integer(a[2]));
    } else {
        w = tensor(a[2], "w");
        if (w.dim() != 2) refuse(PyExc_ValueError, "%s must be [T, K]", "w");
        K = slots_a_token(w.size(1));
    }
    one_device({z, "z"}, {{map, "row_of_slot"}, {w, "w"}, {res, "residual"}, {given, "y"}}, a[5]);
    const Rows rz = rows_of(z, "z");
    sorted_rows(z, z, rz.d, "z");
    const int64_t T = map.numel() / K;
    const int32_t *pm = slots_of(map, T * K);
    const float *pw = w.defined() ? stat_of(w, T * K, "w") : nullptr;
    const OnStream stream(a[5], z);
    Rows rr{};
    if (res.defined()) rr = sorted_rows(res, z, rz.d, "residual");
    const at::Tensor y = given.defined() ? given : fresh({T, rz.d}, z.scalar_type(), z);
    const Rows ry = sorted_rows(y, z, rz.d, "y");
    if (ry.T != T || (res.defined() && rr.T != T))
        refuse(PyExc_ValueError, "%s must have one row a token", ry.T != T ? "y" : "residual");
    check("moe_combine_weighted",
          moe_combine_weighted(rz.p, rz.ld, rz.T, pm, pw, rr.p, rr.ld, T, K, (int)rz.d, dtype(z), ry.p, ry.ld,
                               stream));
    return wrap(y);
}

// dy, z, row_of_slot, w, dz, stream
PyObject *combine_weighted_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 6);
    const at::Tensor dy = tensor(a[0], "dy"), z = tensor(a[1], "z"), map = tensor(a[2], "row_of_slot"),
                     w = tensor(a[3], "w"), given = optional_tensor(a[4], "dz");
    one_device({dy, "dy"}, {{z, "z"}, {map, "row_of_slot"}, {w, "w"}, {given, "dz"}}, a[5]);
    if (w.dim() != 2) refuse(PyExc_ValueError, "%s must be [T, K]", "w");
    const int K = slots_a_token(w.size(1));
    const Rows rdy = rows_of(dy, "dy"), rz = sorted_rows(z, dy, rdy.d, "z");
    const int64_t T = rdy.T;
    const int32_t *pm = slots_of(map, T * K);
    const float *pw = stat_of(w, T * K, "w");
    const OnStream stream(a[5], dy);
    const at::Tensor dz = given.defined() ? given : fresh({rz.T, rz.d}, z.scalar_type(), z);
    const Rows rdz = sorted_rows(dz, dy, rdy.d, "dz");
    if (rdz.T != rz.T) refuse(PyExc_ValueError, "%s must have z's shape", "dz");
    const at::Tensor dw = fresh({T, K}, at::kFloat, dy);
    check("moe_combine_weighted_backward",
          moe_combine_weighted_backward(rdy.p, rdy.ld, rz.p, rz.ld, rz.T, pm, pw, T, K, (int)rz.d, dtype(z),
                                        rdz.p, rdz.ld, static_cast<float *>(dw.data_ptr()), stream));
    return wrap_all(dz, dw);
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

// A projection's operands.
struct Linear {
    at::Tensor x, W, bias, res, ws;
    int T, k, n;
    void *px, *pw, *pb, *pws;
    at::ScalarType type;
    std::vector<int64_t> out;  // the result's shape
};
Linear linear_args(PyObject *x, PyObject *W, PyObject *bias, PyObject *res, PyObject *ws, PyObject *stream) {
    Linear f{tensor(x, "x"), tensor(W, "W"), optional_tensor(bias, "bias"), optional_tensor(res, "residual"),
             tensor(ws, "ws")};
    one_device({f.x, "x"}, {{f.W, "W"}, {f.bias, "bias"}, {f.res, "residual"}, {f.ws, "ws"}}, stream);
    if (f.x.dim() < 1 || f.W.dim() != 2 || f.x.size(-1) != f.W.size(0))
        refuse(PyExc_ValueError, "%s must be [..., k] and W [k, n]", "x");
    f.type = f.x.scalar_type();
    if (f.type != at::kBFloat16 && f.type != at::kHalf)
        refuse(PyExc_TypeError, "a projection takes bf16 or fp16 %s", "x");
    const int64_t k = f.W.size(0), n = f.W.size(1), T = k > 0 ? f.x.numel() / k : 0;
    if (T > INT32_MAX || k > INT32_MAX || n > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", "x");
    f.px = dense(f.x, f.x.sizes(), f.type, "x");
    f.pw = dense(f.W, {k, n}, f.type, "W");
    f.pb = vec_of(f.bias, n, f.x, "bias");
    if (!f.ws.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "ws");
    f.pws = f.ws.data_ptr();
    f.T = (int)T;
    f.k = (int)k;
    f.n = (int)n;
    f.out = f.x.sizes().vec();
    f.out.back() = n;
    return f;
}
moe_dtype_t bias_type(const Linear &f) { return dtype(f.bias.defined() ? f.bias : f.x); }

// x, W, bias, act, residual, ws, Y, stream
PyObject *linear(PyObject *const *a, Py_ssize_t n) {
    expect(n, 8);
    const Linear f = linear_args(a[0], a[1], a[2], a[4], a[5], a[7]);
    const at::Tensor given = optional_tensor(a[6], "Y");
    one_device({f.x, "x"}, {{given, "Y"}}, Py_None);
    const OnStream stream(a[7], f.x);
    const at::Tensor Y = given.defined() ? given : fresh(f.out, f.type, f.x);
    void *py = dense(Y, f.out, f.type, "Y"), *pr = f.res.defined() ? dense(f.res, f.out, f.type, "residual") : nullptr;
    check("moe_linear_forward",
          moe_linear_forward(f.px, f.pw, f.pb, pr, f.T, f.k, f.n, (moe_act_t)integer(a[3]), dtype(f.x), bias_type(f),
                             py, f.pws, f.ws.nbytes(), stream));
    return wrap(Y);
}

// x, W, bias, act, residual, ws, stream
PyObject *linear_train(PyObject *const *a, Py_ssize_t n) {
    expect(n, 7);
    const Linear f = linear_args(a[0], a[1], a[2], a[4], a[5], a[6]);
    const OnStream stream(a[6], f.x);
    const moe_act_t act = (moe_act_t)integer(a[3]);
    void *pr = f.res.defined() ? dense(f.res, f.out, f.type, "residual") : nullptr;
    const at::Tensor Y = fresh(f.out, f.type, f.x);
    at::Tensor F;
    if (act != MOE_ACT_NONE) F = fresh({(int64_t)moe_ffn_saved_floats(f.T, f.n)}, at::kFloat, f.x);
    check("moe_linear_forward_train",
          moe_linear_forward_train(f.px, f.pw, f.pb, pr, f.T, f.k, f.n, act, dtype(f.x), bias_type(f), Y.data_ptr(),
                                   F.defined() ? static_cast<float *>(F.data_ptr()) : nullptr, f.pws, f.ws.nbytes(), stream));
    return wrap_all(Y, F);
}

// dY, x, W, F, fp32 bias gradient or not (None: no bias gradient), need_dx, need_dw, ws, stream
PyObject *linear_backward(PyObject *const *a, Py_ssize_t n) {
    expect(n, 9);
    const Linear f = linear_args(a[1], a[2], Py_None, Py_None, a[7], a[8]);
    const at::Tensor dY = tensor(a[0], "dY"), F = optional_tensor(a[3], "F");
    one_device({f.x, "x"}, {{dY, "dY"}, {F, "F"}}, Py_None);
    const OnStream stream(a[8], f.x);
    void *pdy = dense(dY, f.out, f.type, "dY");
    const float *pf = F.defined() ? static_cast<const float *>(
                                        dense(F, {(int64_t)moe_ffn_saved_floats(f.T, f.n)}, at::kFloat, "F"))
                                  : nullptr;
    const bool db = a[4] != Py_None, b32 = db && truth(a[4]);
    at::Tensor dX, dW, dbias;
    if (truth(a[5])) dX = fresh(f.x.sizes(), f.type, f.x);
    if (truth(a[6])) dW = fresh({f.k, f.n}, f.type, f.x);
    if (db) dbias = fresh({f.n}, b32 ? at::kFloat : f.type, f.x);
    auto data = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    check("moe_linear_backward",
          moe_linear_backward(pdy, f.px, f.pw, pf, f.T, f.k, f.n, dtype(f.x), b32 ? MOE_DTYPE_F32 : dtype(f.x),
                              data(dX), data(dW), data(dbias), f.pws, f.ws.nbytes(), stream));
    return wrap_all(dX, dW, dbias);
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
                           MOE_ENTRY(ffn_backward), MOE_ENTRY(linear), MOE_ENTRY(linear_train),
                           MOE_ENTRY(linear_backward), MOE_ENTRY(block_norm),
                           MOE_ENTRY(block_norm_backward), MOE_ENTRY(dispatch),
                           MOE_ENTRY(combine_weighted), MOE_ENTRY(combine_weighted_backward),
                           MOE_ENTRY(set_error),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
