// C ABI of the sub-block operators around the layer (layer norm, residual dropout, dense gated
// feed-forward block, projections, norms around a block, dispatch and combine): argument checks
// and launches. Errors are returned before anything is enqueued.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "common.cuh"

using namespace moe;

namespace {

bool valid_type(moe_dtype_t t) {
    return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32;
}
int size_of(moe_dtype_t t) { return t == MOE_DTYPE_F32 ? 4 : 2; }
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A [T,d] matrix of the operators: whole elements, rows that do not overlap, and
// offsets that 64 bits hold.
moe_status_t check_matrix(const void *p, int64_t ld, int64_t T, int d, moe_dtype_t t) {
    if (p == nullptr || !aligned(p, size_of(t))) return MOE_ERR_INVALID_ARG;
    if (ld < d && T > 1) return MOE_ERR_INVALID_ARG;
    if (T > 1 && ld > (1ll << 58) / T) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status_t check_shape(int64_t T, int d, moe_dtype_t t) {
    if (T < 0 || d < 1 || !valid_type(t)) return MOE_ERR_INVALID_ARG;
    if (T > (1ll << 58) / d) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// An output in the place of an operand has its row stride: with another one, rows would be
// overwritten before they are read.
bool strides_clash(const void *in, int64_t ldin, const void *out, int64_t ldout, int64_t T) {
    return in == out && ldin != ldout && T > 1;
}

moe_status_t drop(const void *x, int64_t ldx, const void *res, int64_t ldr, int64_t T, int d,
                  double p, uint64_t seed, uint64_t offset, const uint64_t *offset_dev,
                  moe_dtype_t type, void *y, int64_t ldy, void *stream) {
    moe_status_t st = check_shape(T, d, type);
    if (st != MOE_OK) return st;
    if (!(p >= 0.0 && p <= 1.0) || !aligned(offset_dev, 8)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if ((st = check_matrix(x, ldx, T, d, type)) != MOE_OK) return st;
    if ((st = check_matrix(y, ldy, T, d, type)) != MOE_OK) return st;
    if (res != nullptr && (st = check_matrix(res, ldr, T, d, type)) != MOE_OK) return st;
    if (strides_clash(x, ldx, y, ldy, T) || strides_clash(res, ldr, y, ldy, T)) return MOE_ERR_INVALID_ARG;
    if ((st = check_arch()) != MOE_OK) return st;
    const uint32_t thr = (uint32_t)floor(p * 65536.0 + 0.5);
    return from_cuda(launch_dropout(x, ldx, res, ldr, y, ldy, T, d, thr, seed, offset, offset_dev,
                                    type, as_stream(stream)));
}

// The shape of a map of T x K slots onto `rows` sorted rows of d elements.
moe_status_t check_slots(const int32_t *row_of_slot, int64_t T, int K, int d, int64_t rows,
                         moe_dtype_t type) {
    moe_status_t st = check_shape(T, d, type);
    if (st != MOE_OK) return st;
    if (K < 1 || rows < 0 || !aligned(row_of_slot, 4) || (row_of_slot == nullptr && T > 0))
        return MOE_ERR_INVALID_ARG;
    // (columns are counted in 32 bits, a step past the last one too)
    if (K > kMaxK || T > INT32_MAX / K || d > kMaxRowWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}
// A matrix of sorted rows; there may be none of them.
moe_status_t check_sorted(const void *p, int64_t ld, int64_t rows, int d, moe_dtype_t type) {
    return rows == 0 ? MOE_OK : check_matrix(p, ld, rows, d, type);
}

// The row that this thread's next layer norm withholds (moe_selftest_layernorm_withhold).
thread_local int64_t t_withheld = -1;
int64_t take_withheld() {
    const int64_t row = t_withheld;
    t_withheld = -1;
    return row;
}

// ---- norms around a block

// What forward and backward refuse alike of the operands that both have.
moe_status_t check_block_norm(const BlockNormCall &c, moe_gate_t kind, int norms, moe_dtype_t wtype) {
    const moe_status_t st = check_shape(c.T, c.d, c.type);
    if (st != MOE_OK) return st;
    if (c.d > kBlockNormMaxWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((wtype != c.type && wtype != MOE_DTYPE_F32) || (norms & ~(MOE_NORM_POST | MOE_NORM_PRE)) != 0 ||
        (kind != MOE_GATE_NONE && kind != MOE_GATE_ROW && kind != MOE_GATE_FULL) ||
        (kind == MOE_GATE_NONE && c.gate.p != nullptr) || !(c.scale == c.scale))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(c.post, size_of(wtype)) || !aligned(c.pre, size_of(wtype)) || !aligned(c.r_post, 4) ||
        !aligned(c.r_pre, 4))
        return MOE_ERR_INVALID_ARG;
    if (!c.pre_norm && c.pre != nullptr) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}
bool plain_norm(const BlockNormCall &c, moe_gate_t kind) {
    return kind == MOE_GATE_NONE && !c.post_norm && c.pre_norm && c.post == nullptr && c.scale == 1.f;
}
// The call's matrices: each one there, and no output with another stride in an input's place
// or in another output's.
moe_status_t check_matrices(const BlockNormCall &c, std::initializer_list<Matrix> in,
                            std::initializer_list<Matrix> out) {
    moe_status_t st;
    for (const Matrix &m : in)
        if ((st = check_matrix(m.p, m.ld, c.T, c.d, c.type)) != MOE_OK) return st;
    for (const Matrix *o = out.begin(); o != out.end(); ++o) {
        if ((st = check_matrix(o->p, o->ld, c.T, c.d, c.type)) != MOE_OK) return st;
        for (const Matrix &m : in)
            if (strides_clash(m.p, m.ld, o->p, o->ld, c.T)) return MOE_ERR_INVALID_ARG;
        for (const Matrix *q = out.begin(); q != o; ++q)
            if (q->p == o->p) return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}
// Matrix `m` if the call has one, else another that is checked all the same.
Matrix if_any(bool has, const Matrix &m, const Matrix &other) { return has ? m : other; }

// ---- dense feed-forward block

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

moe_status_t check_ffn(int T, int d, int n, moe_act_t act, moe_dtype_t type) {
    if (T < 0 || d < 1 || n < 1 || !valid_type(type) ||
        (act != MOE_ACT_SILU && act != MOE_ACT_GELU_TANH))
        return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0 || n % 8 != 0 || d > kFfnMaxWidth || n > kFfnMaxWidth || type == MOE_DTYPE_F32)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    // row tiles and columns of every product stay within 32-bit indices
    if (T > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// Regions behind the control words: the backward's dA1, dA3, or H of a forward
// without saved tensors; then the parts of cut tiles.
struct FfnWs {
    size_t h, part, da1, da3, total;
};
FfnWs ffn_ws(int T, int d, int n, bool train) {
    FfnWs w;
    const size_t act = align256((size_t)T * n * 2);
    w.h = w.da1 = align256(kFfnControlBytes);
    w.da3 = w.da1 + act;
    w.part = train ? w.da3 + act : w.h + act;
    const bool tiled = train || !ffn_streams(T, d, n);
    w.total = w.part + (tiled ? align256(ffn_dense_part_bytes()) : 0);
    // a workspace for T tokens serves fewer, whichever kernel they take
    const int few = std::min(T, kFfnStreamTokens);
    w.total = std::max(w.total, w.h + align256((size_t)few * n * 2) +
                                    align256(ffn_stream_part_bytes(few, d, n)));
    return w;
}
// The same for projections: the training's dA, the sums of its bias' gradient, then the parts.
struct LinearWs {
    size_t da, sums, part, total;
};
LinearWs linear_ws(int T, int k, int n, bool train) {
    LinearWs w;
    w.da = align256(kFfnControlBytes);
    w.sums = w.da + (train ? align256((size_t)T * n * 2) : 0);
    w.part = w.sums + (train ? align256((size_t)linear_sum_rows(T, n) * n * sizeof(float)) : 0);
    const bool tiled = train || !linear_streams(T, n);
    w.total = w.part + (tiled ? align256(ffn_dense_part_bytes()) : 0);
    // a workspace for T tokens serves fewer, whichever kernel they take
    const int few = std::min(T, kFfnStreamTokens);
    w.total = std::max(w.total, w.part + align256(linear_stream_part_bytes(few, k, n)));
    return w;
}
moe_status_t check_linear(int T, int k, int n, moe_act_t act, moe_dtype_t type, moe_dtype_t btype) {
    const moe_status_t st =
        check_ffn(T, k, n, act == MOE_ACT_NONE ? MOE_ACT_SILU : act, type);
    if (st != MOE_OK) return st;
    return btype == type || btype == MOE_DTYPE_F32 ? MOE_OK : MOE_ERR_INVALID_ARG;
}
moe_status_t check_linear_ws(void *ws, size_t ws_bytes, int T, int k, int n, bool train) {
    if (ws == nullptr || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    return ws_bytes < linear_ws(T, k, n, train).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

char *at(void *ws, size_t off) { return static_cast<char *>(ws) + off; }

// A dense operand's bytes; none where p is NULL.
struct Span {
    uintptr_t at, end;
    Span(const void *p, size_t bytes)
        : at(reinterpret_cast<uintptr_t>(p)), end(p == nullptr ? at : at + bytes) {}
};
// Whether one of the outputs shares bytes with an operand or with another output.
bool overlaps(std::initializer_list<Span> in, std::initializer_list<Span> out) {
    auto shares = [](const Span &a, const Span &b) { return a.at < b.end && b.at < a.end; };
    for (const Span *o = out.begin(); o != out.end(); ++o) {
        for (const Span &i : in)
            if (shares(i, *o)) return true;
        for (const Span *q = out.begin(); q != o; ++q)
            if (shares(*q, *o)) return true;
    }
    return false;
}

bool all_aligned16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr || !aligned(p, 16)) return false;
    return true;
}

moe_status_t check_ffn_ws(void *ws, size_t ws_bytes, int T, int d, int n, bool train) {
    if (ws == nullptr || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    return ws_bytes < ffn_ws(T, d, n, train).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_layernorm_forward(const void *x, int64_t ldx, const void *gamma,
                                   const void *beta, int64_t T, int d, float eps,
                                   moe_dtype_t type, moe_dtype_t wtype, void *y, int64_t ldy,
                                   float *mean, float *rstd, void *stream) {
    moe_status_t st = check_shape(T, d, type);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.f) || (wtype != type && wtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
    if (!aligned(gamma, size_of(wtype)) || !aligned(beta, size_of(wtype)) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if ((st = check_matrix(x, ldx, T, d, type)) != MOE_OK) return st;
    if ((st = check_matrix(y, ldy, T, d, type)) != MOE_OK) return st;
    if (strides_clash(x, ldx, y, ldy, T)) return MOE_ERR_INVALID_ARG;
    if ((st = check_arch()) != MOE_OK) return st;
    return from_cuda(launch_layernorm_forward(x, ldx, gamma, beta, y, ldy, mean, rstd, T, d, eps,
                                              type, wtype == MOE_DTYPE_F32, take_withheld(),
                                              as_stream(stream)));
}

size_t moe_layernorm_scratch_bytes(int64_t T, int d) {
    if (T < 0 || d < 1) return 0;
    return ((size_t)ln_partials(T) * 2 * (size_t)d * sizeof(float) + 255) / 256 * 256;
}

moe_status_t moe_layernorm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                    const void *gamma, const float *mean, const float *rstd,
                                    const void *dres, int64_t lddres, int64_t T, int d,
                                    moe_dtype_t type, moe_dtype_t wtype, void *dx, int64_t lddx,
                                    void *dgamma, void *dbeta, void *scratch,
                                    size_t scratch_bytes, void *stream) {
    moe_status_t st = check_shape(T, d, type);
    if (st != MOE_OK) return st;
    if (wtype != type && wtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    const int ws = size_of(wtype);
    if (!aligned(gamma, ws) || !aligned(dgamma, ws) || !aligned(dbeta, ws))
        return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (mean == nullptr || rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4))
            return MOE_ERR_INVALID_ARG;
        if ((st = check_matrix(dy, lddy, T, d, type)) != MOE_OK) return st;
        if ((st = check_matrix(x, ldx, T, d, type)) != MOE_OK) return st;
        if ((st = check_matrix(dx, lddx, T, d, type)) != MOE_OK) return st;
        if (dres != nullptr && (st = check_matrix(dres, lddres, T, d, type)) != MOE_OK) return st;
        if (strides_clash(dy, lddy, dx, lddx, T) || strides_clash(x, ldx, dx, lddx, T) ||
            strides_clash(dres, lddres, dx, lddx, T))
            return MOE_ERR_INVALID_ARG;
        if (dgamma != nullptr || dbeta != nullptr) {
            if (scratch == nullptr || !aligned(scratch, 256)) return MOE_ERR_INVALID_ARG;
            if (scratch_bytes < moe_layernorm_scratch_bytes(T, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        }
    }
    if ((st = check_arch()) != MOE_OK) return st;
    if (T == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        if (dgamma != nullptr) e = cudaMemsetAsync(dgamma, 0, (size_t)d * ws, as_stream(stream));
        if (e == cudaSuccess && dbeta != nullptr)
            e = cudaMemsetAsync(dbeta, 0, (size_t)d * ws, as_stream(stream));
        return from_cuda(e);
    }
    return from_cuda(launch_layernorm_backward(dy, lddy, x, ldx, gamma, mean, rstd, dres, lddres,
                                               dx, lddx, dgamma, dbeta, T, d, type,
                                               wtype == MOE_DTYPE_F32,
                                               static_cast<float *>(scratch), take_withheld(),
                                               as_stream(stream)));
}

moe_status_t moe_selftest_layernorm_withhold(int64_t row) {
    t_withheld = row >= 0 ? row : -1;
    return MOE_OK;
}

moe_status_t moe_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                         int64_t T, int d, double p, uint64_t seed, uint64_t offset,
                         const uint64_t *offset_dev, moe_dtype_t type, void *y, int64_t ldy,
                         void *stream) {
    return drop(x, ldx, residual, ldr, T, d, p, seed, offset, offset_dev, type, y, ldy, stream);
}

moe_status_t moe_dropout_backward(const void *dy, int64_t lddy, int64_t T, int d, double p,
                                  uint64_t seed, uint64_t offset, const uint64_t *offset_dev,
                                  moe_dtype_t type, void *dx, int64_t lddx, void *stream) {
    return drop(dy, lddy, nullptr, 0, T, d, p, seed, offset, offset_dev, type, dx, lddx, stream);
}

size_t moe_linear_workspace_bytes(int T, int k, int n, int train) {
    if (check_linear(T, k, n, MOE_ACT_NONE, MOE_DTYPE_BF16, MOE_DTYPE_BF16) != MOE_OK) return 0;
    return linear_ws(T, k, n, train != 0).total;
}

static moe_status_t linear_forward(const void *X, const void *W, const void *bias, const void *residual,
                                   int T, int k, int n, moe_act_t act, moe_dtype_t type,
                                   moe_dtype_t btype, void *Y, float *F, bool train, void *ws,
                                   size_t ws_bytes, void *stream) {
    moe_status_t st = check_linear(T, k, n, act, type, btype);
    if (st != MOE_OK || T == 0) return st;
    if (!all_aligned16({X, W, Y}) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(F, 16) ||
        (train && (F != nullptr) != (act != MOE_ACT_NONE)))
        return MOE_ERR_INVALID_ARG;
    // Y and F are stored while other tiles read their operands: of all of them, only the residual is
    // read where it is overwritten
    const size_t rows = T;
    const Span y(Y, rows * n * 2), f(F, moe_ffn_saved_floats(T, n) * sizeof(float)), x(X, rows * k * 2),
        w(W, (size_t)k * n * 2), b(bias, (size_t)n * size_of(btype)), r(residual, rows * n * 2);
    if (overlaps({x, w, b}, {y, f}) || overlaps({r}, {f}) || (residual != Y && overlaps({r}, {y})))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_linear_ws(ws, ws_bytes, T, k, n, train)) != MOE_OK) return st;
    if ((st = check_arch()) != MOE_OK) return st;
    const LinearCall c{X, W, bias, residual, Y, T, k, n, act, type == MOE_DTYPE_F16, btype == MOE_DTYPE_F32};
    void *part = at(ws, linear_ws(T, k, n, train).part);
    uint32_t *ticket = reinterpret_cast<uint32_t *>(at(ws, kFfnTicketOffset));
    uint32_t *err = static_cast<uint32_t *>(ws);
    cudaStream_t s = as_stream(stream);
    if (F == nullptr && linear_streams(T, n))
        return from_cuda(launch_linear_stream(c, static_cast<float *>(part), ticket, err, s));
    return from_cuda(launch_linear_tiled(c, F, static_cast<float4 *>(part), ticket, err, s));
}

moe_status_t moe_linear_forward(const void *X, const void *W, const void *bias,
                                const void *residual, int T, int k, int n, moe_act_t act,
                                moe_dtype_t type, moe_dtype_t btype, void *Y, void *ws,
                                size_t ws_bytes, void *stream) {
    return linear_forward(X, W, bias, residual, T, k, n, act, type, btype, Y, nullptr, false, ws, ws_bytes,
                          stream);
}

moe_status_t moe_linear_forward_train(const void *X, const void *W, const void *bias,
                                      const void *residual, int T, int k, int n, moe_act_t act,
                                      moe_dtype_t type, moe_dtype_t btype, void *Y, float *F,
                                      void *ws, size_t ws_bytes, void *stream) {
    return linear_forward(X, W, bias, residual, T, k, n, act, type, btype, Y, F, true, ws, ws_bytes, stream);
}

moe_status_t moe_linear_backward(const void *dY, const void *X, const void *W, const float *F, int T,
                                 int k, int n, moe_dtype_t type, moe_dtype_t btype, void *dX,
                                 void *dW, void *dbias, void *ws, size_t ws_bytes, void *stream) {
    moe_status_t st = check_linear(T, k, n, MOE_ACT_NONE, type, btype);
    if (st != MOE_OK) return st;
    if (!aligned(dX, 16) || !aligned(dW, 16) || !aligned(dbias, size_of(btype))) return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!all_aligned16({dY}) || !aligned(F, 16) || (dX != nullptr && !all_aligned16({W})) ||
            (dW != nullptr && !all_aligned16({X})))
            return MOE_ERR_INVALID_ARG;
        const size_t rows = T;
        const Span dy(dY, rows * n * 2), f(F, moe_ffn_saved_floats(T, n) * sizeof(float)), x(X, rows * k * 2),
            wt(W, (size_t)k * n * 2), dx(dX, rows * k * 2), dw(dW, (size_t)k * n * 2),
            db(dbias, (size_t)n * size_of(btype));
        if (overlaps({dy, f, x, wt}, {dx, dw, db})) return MOE_ERR_INVALID_ARG;
        if ((st = check_linear_ws(ws, ws_bytes, T, k, n, true)) != MOE_OK) return st;
    }
    if ((st = check_arch()) != MOE_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (T == 0) {  // sums over no tokens
        cudaError_t e = cudaSuccess;
        if (dW != nullptr) e = cudaMemsetAsync(dW, 0, (size_t)k * n * 2, s);
        if (dbias != nullptr && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)n * size_of(btype), s);
        return from_cuda(e);
    }
    const LinearWs w = linear_ws(T, k, n, true);
    const bool f16 = type == MOE_DTYPE_F16;
    const bool products = dX != nullptr || dW != nullptr;
    void *dA = F != nullptr ? at(ws, w.da) : const_cast<void *>(dY);
    if (!products && dbias == nullptr) return MOE_OK;
    float *sums = dbias != nullptr ? reinterpret_cast<float *>(at(ws, w.sums)) : nullptr;
    const bool b32 = btype == MOE_DTYPE_F32;
    cudaError_t e = launch_linear_grad(dY, F, T, n, f16, dA, sums, s);
    const bool beside = dW != nullptr && linear_sum_rows(T, n) <= kLinearSumsBeside;
    if (e == cudaSuccess && dbias != nullptr && !beside)
        e = launch_linear_bias(sums, T, n, f16, dbias, b32, s);
    if (e == cudaSuccess)
        e = launch_linear_products(dA, X, W, T, k, n, f16, dX, dW, beside ? dbias : nullptr, b32, sums,
                                   reinterpret_cast<float4 *>(at(ws, w.part)),
                                   reinterpret_cast<uint32_t *>(at(ws, kFfnTicketOffset)),
                                   static_cast<uint32_t *>(ws), s);
    return from_cuda(e);
}

size_t moe_block_norm_scratch_bytes(int64_t T, int d) {
    if (T < 0 || d < 1) return 0;
    return align256((size_t)block_norm_partials(T) * 2 * (size_t)d * sizeof(float));
}

moe_status_t moe_block_norm_forward(const void *x, int64_t ldx, const void *b, int64_t ldb,
                                    const void *gate, int64_t ldgate, moe_gate_t gate_kind,
                                    const void *post, const void *pre, float scale, int norms,
                                    int64_t T, int d, float eps, moe_dtype_t type,
                                    moe_dtype_t wtype, void *y, int64_t ldy, void *u, int64_t ldu,
                                    float *rstd_post, float *rstd_pre, void *stream) {
    BlockNormCall c{};
    c.x = {x, ldx};
    c.b = {b, ldb};
    c.gate = {gate, ldgate};
    c.y = {y, ldy};
    c.u = {u, ldu};
    c.post = post;
    c.pre = pre;
    c.r_post = rstd_post;
    c.r_pre = rstd_pre;
    c.T = T;
    c.d = d;
    c.type = type;
    c.w32 = wtype == MOE_DTYPE_F32;
    c.gate_rows = gate_kind == MOE_GATE_FULL;
    c.post_norm = (norms & MOE_NORM_POST) != 0;
    c.pre_norm = (norms & MOE_NORM_PRE) != 0;
    c.scale = scale;
    c.eps = eps;
    moe_status_t st = check_block_norm(c, gate_kind, norms, wtype);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.f) || (!c.pre_norm && u != nullptr)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const bool full = gate_kind == MOE_GATE_FULL;
    if (b == nullptr) {
        if (!plain_norm(c, gate_kind) || y != nullptr) return MOE_ERR_INVALID_ARG;
        st = check_matrices(c, {c.x}, {c.u});
    } else {
        if (gate_kind == MOE_GATE_ROW && (gate == nullptr || !aligned(gate, 4))) return MOE_ERR_INVALID_ARG;
        const std::initializer_list<Matrix> in = {c.x, c.b, if_any(full, c.gate, c.x)};
        st = c.pre_norm ? check_matrices(c, in, {c.y, c.u}) : check_matrices(c, in, {c.y});
    }
    if (st != MOE_OK || (st = check_arch()) != MOE_OK) return st;
    return from_cuda(launch_block_norm_forward(c, take_withheld(), as_stream(stream)));
}

moe_status_t moe_block_norm_backward(const void *dy, int64_t lddy, const void *du, int64_t lddu,
                                     const void *x, int64_t ldx, const void *b, int64_t ldb,
                                     const void *gate, int64_t ldgate, moe_gate_t gate_kind,
                                     const void *post, const void *pre, float scale, int norms,
                                     const float *rstd_post, const float *rstd_pre, int64_t T, int d,
                                     moe_dtype_t type, moe_dtype_t wtype, void *dx, int64_t lddx,
                                     void *db, int64_t lddb, void *dgate, int64_t lddgate,
                                     void *dpost, void *dpre, void *scratch, size_t scratch_bytes,
                                     void *stream) {
    BlockNormCall c{};
    c.x = {x, ldx};
    c.b = {b, ldb};
    c.gate = {gate, ldgate};
    c.post = post;
    c.pre = pre;
    c.r_post = const_cast<float *>(rstd_post);
    c.r_pre = const_cast<float *>(rstd_pre);
    c.T = T;
    c.d = d;
    c.type = type;
    c.w32 = wtype == MOE_DTYPE_F32;
    c.gate_rows = gate_kind == MOE_GATE_FULL;
    c.post_norm = (norms & MOE_NORM_POST) != 0;
    c.pre_norm = (norms & MOE_NORM_PRE) != 0;
    c.scale = scale;
    c.dy = {dy, lddy};
    c.du = {du, lddu};
    c.dx = {dx, lddx};
    c.db = {db, lddb};
    c.dgate = {dgate, lddgate};
    c.dpost = dpost;
    c.dpre = dpre;
    c.part = static_cast<float *>(scratch);
    moe_status_t st = check_block_norm(c, gate_kind, norms, wtype);
    if (st != MOE_OK) return st;
    const int ws = size_of(wtype);
    if (!aligned(dpost, ws) || !aligned(dpre, ws) || (!c.pre_norm && (du != nullptr || dpre != nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        const bool full = gate_kind == MOE_GATE_FULL;
        if ((dy == nullptr && !c.pre_norm) || (c.post_norm && rstd_post == nullptr) ||
            (c.pre_norm && rstd_pre == nullptr))
            return MOE_ERR_INVALID_ARG;
        const Matrix g = if_any(full, c.gate, c.x), u = if_any(c.pre_norm, c.du, c.x),
                     s = if_any(dy != nullptr, c.dy, c.x);
        if (b == nullptr) {
            if (!plain_norm(c, gate_kind) || db != nullptr || dgate != nullptr || dpost != nullptr)
                return MOE_ERR_INVALID_ARG;
            st = check_matrices(c, {c.x, u, s}, {c.dx});
        } else {
            if (gate_kind == MOE_GATE_ROW &&
                (gate == nullptr || dgate == nullptr || !aligned(gate, 4) || !aligned(dgate, 4)))
                return MOE_ERR_INVALID_ARG;
            if (gate_kind == MOE_GATE_NONE && dgate != nullptr) return MOE_ERR_INVALID_ARG;
            const std::initializer_list<Matrix> in = {c.x, c.b, g, u, s};
            st = full ? check_matrices(c, in, {c.dx, c.db, c.dgate}) : check_matrices(c, in, {c.dx, c.db});
        }
        if (st != MOE_OK) return st;
        if (dpost != nullptr || dpre != nullptr) {
            if (scratch == nullptr || !aligned(scratch, 256)) return MOE_ERR_INVALID_ARG;
            if (scratch_bytes < moe_block_norm_scratch_bytes(T, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        }
    }
    if ((st = check_arch()) != MOE_OK) return st;
    if (T == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        for (void *p : {dpost, dpre})
            if (p != nullptr && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)d * ws, as_stream(stream));
        return from_cuda(e);
    }
    return from_cuda(launch_block_norm_backward(c, take_withheld(), as_stream(stream)));
}

moe_status_t moe_dispatch(const void *x, int64_t ldx, const int32_t *row_of_slot, int64_t T, int K,
                          int d, moe_dtype_t type, void *xg, int64_t ldxg, int64_t rows,
                          void *stream) {
    moe_status_t st = check_slots(row_of_slot, T, K, d, rows, type);
    if (st != MOE_OK || T == 0) return st;
    if ((st = check_matrix(x, ldx, T, d, type)) != MOE_OK) return st;
    if ((st = check_sorted(xg, ldxg, rows, d, type)) != MOE_OK) return st;
    if (x == xg) return MOE_ERR_INVALID_ARG;
    if ((st = check_arch()) != MOE_OK || rows == 0) return st;
    RowArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.row_of_slot = row_of_slot;
    a.out = xg;
    a.ldo = ldxg;
    a.T = T;
    a.rows = rows;
    a.K = K;
    a.d = d;
    return from_cuda(launch_dispatch(a, type, as_stream(stream)));
}

moe_status_t moe_combine_weighted(const void *z, int64_t ldz, int64_t rows,
                                  const int32_t *row_of_slot, const float *w, const void *residual,
                                  int64_t ldr, int64_t T, int K, int d, moe_dtype_t type, void *y,
                                  int64_t ldy, void *stream) {
    moe_status_t st = check_slots(row_of_slot, T, K, d, rows, type);
    if (st != MOE_OK) return st;
    if (!aligned(w, 4)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if ((st = check_sorted(z, ldz, rows, d, type)) != MOE_OK) return st;
    if ((st = check_matrix(y, ldy, T, d, type)) != MOE_OK) return st;
    if (residual != nullptr && (st = check_matrix(residual, ldr, T, d, type)) != MOE_OK) return st;
    if (z == y || strides_clash(residual, ldr, y, ldy, T)) return MOE_ERR_INVALID_ARG;
    if ((st = check_arch()) != MOE_OK) return st;
    RowArgs a{};
    a.z = z;
    a.ldz = ldz;
    a.rows = rows;
    a.row_of_slot = row_of_slot;
    a.w = w;
    a.res = residual;
    a.ldr = ldr;
    a.out = y;
    a.ldo = ldy;
    a.T = T;
    a.K = K;
    a.d = d;
    return from_cuda(launch_sum_rows(a, type, as_stream(stream)));
}

moe_status_t moe_combine_weighted_backward(const void *dy, int64_t lddy, const void *z, int64_t ldz,
                                           int64_t rows, const int32_t *row_of_slot, const float *w,
                                           int64_t T, int K, int d, moe_dtype_t type, void *dz,
                                           int64_t lddz, float *dw, void *stream) {
    moe_status_t st = check_slots(row_of_slot, T, K, d, rows, type);
    if (st != MOE_OK || T == 0) return st;
    if (w == nullptr || dw == nullptr || !aligned(w, 4) || !aligned(dw, 4)) return MOE_ERR_INVALID_ARG;
    if ((st = check_matrix(dy, lddy, T, d, type)) != MOE_OK) return st;
    if ((st = check_sorted(z, ldz, rows, d, type)) != MOE_OK) return st;
    if ((st = check_sorted(dz, lddz, rows, d, type)) != MOE_OK) return st;
    if (dy == dz || strides_clash(z, ldz, dz, lddz, rows)) return MOE_ERR_INVALID_ARG;
    if ((st = check_arch()) != MOE_OK) return st;
    RowArgs a{};
    a.x = dy;
    a.ldx = lddy;
    a.z = z;
    a.ldz = ldz;
    a.rows = rows;
    a.row_of_slot = row_of_slot;
    a.w = w;
    a.out = dz;
    a.ldo = lddz;
    a.dw = dw;
    a.T = T;
    a.K = K;
    a.d = d;
    return from_cuda(launch_combine_backward(a, type, as_stream(stream)));
}

size_t moe_ffn_workspace_bytes(int T, int d, int n, int train) {
    if (check_ffn(T, d, n, MOE_ACT_SILU, MOE_DTYPE_BF16) != MOE_OK) return 0;
    return ffn_ws(T, d, n, train != 0).total;
}

size_t moe_ffn_saved_floats(int T, int n) {
    if (T < 0 || n < 1) return 0;
    return (size_t)((T + 31ll) / 32) * ((n + 31ll) / 32) * 1024;
}

moe_status_t moe_ffn_workspace_init(void *ws, size_t ws_bytes, void *stream) {
    if (ws == nullptr || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < kFfnControlBytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const moe_status_t st = check_arch();
    if (st != MOE_OK) return st;
    return from_cuda(cudaMemsetAsync(ws, 0, kFfnControlBytes, as_stream(stream)));
}

moe_status_t moe_ffn_forward(const void *X, const void *W1, const void *W3, const void *W2, int T,
                             int d, int n, moe_act_t act, moe_dtype_t type, void *Y, void *ws,
                             size_t ws_bytes, void *stream) {
    moe_status_t st = check_ffn(T, d, n, act, type);
    if (st != MOE_OK || T == 0) return st;
    if (!all_aligned16({X, W1, W3, W2, Y})) return MOE_ERR_INVALID_ARG;
    if ((st = check_ffn_ws(ws, ws_bytes, T, d, n, false)) != MOE_OK) return st;
    if ((st = check_arch()) != MOE_OK) return st;
    const FfnWs w = ffn_ws(T, d, n, false);
    uint32_t *err = static_cast<uint32_t *>(ws);
    uint32_t *ticket = reinterpret_cast<uint32_t *>(at(ws, kFfnTicketOffset));
    float4 *part = reinterpret_cast<float4 *>(at(ws, w.part));
    const bool f16 = type == MOE_DTYPE_F16;
    cudaStream_t s = as_stream(stream);
    if (ffn_streams(T, d, n))
        return from_cuda(launch_ffn_stream(X, W1, W3, W2, T, d, n, act, f16, at(ws, w.h), Y,
                                           reinterpret_cast<float *>(part), ticket, err, s));
    cudaError_t e = launch_ffn_gate(X, W1, W3, T, d, n, act, f16, at(ws, w.h), nullptr, nullptr, part,
                                    ticket, err, s);
    if (e == cudaSuccess) e = launch_ffn_down(at(ws, w.h), W2, T, d, n, f16, Y, part, ticket, err, s);
    return from_cuda(e);
}

moe_status_t moe_ffn_forward_train(const void *X, const void *W1, const void *W3, const void *W2,
                                   int T, int d, int n, moe_act_t act, moe_dtype_t type, void *Y,
                                   void *H, float *F1, float *F3, void *ws, size_t ws_bytes,
                                   void *stream) {
    moe_status_t st = check_ffn(T, d, n, act, type);
    if (st != MOE_OK || T == 0) return st;
    if (!all_aligned16({X, W1, W3, W2, Y, H, F1, F3})) return MOE_ERR_INVALID_ARG;
    if ((st = check_ffn_ws(ws, ws_bytes, T, d, n, true)) != MOE_OK) return st;
    if ((st = check_arch()) != MOE_OK) return st;
    uint32_t *err = static_cast<uint32_t *>(ws);
    uint32_t *ticket = reinterpret_cast<uint32_t *>(at(ws, kFfnTicketOffset));
    float4 *part = reinterpret_cast<float4 *>(at(ws, ffn_ws(T, d, n, true).part));
    const bool f16 = type == MOE_DTYPE_F16;
    cudaStream_t s = as_stream(stream);
    cudaError_t e = launch_ffn_gate(X, W1, W3, T, d, n, act, f16, H, F1, F3, part, ticket, err, s);
    if (e == cudaSuccess) e = launch_ffn_down(H, W2, T, d, n, f16, Y, part, ticket, err, s);
    return from_cuda(e);
}

moe_status_t moe_ffn_backward(const void *dY, const void *X, const void *W1, const void *W3,
                              const void *W2, const void *H, const float *F1, const float *F3,
                              int T, int d, int n, moe_act_t act, moe_dtype_t type, void *dX,
                              void *dW1, void *dW3, void *dW2, void *ws, size_t ws_bytes,
                              void *stream) {
    moe_status_t st = check_ffn(T, d, n, act, type);
    if (st != MOE_OK) return st;
    const int given = (dW1 != nullptr) + (dW3 != nullptr) + (dW2 != nullptr);
    if (given != 0 && (given != 3 || !all_aligned16({dW1, dW3, dW2}))) return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!all_aligned16({dY, X, W1, W3, W2, H, F1, F3}) || !aligned(dX, 16))
            return MOE_ERR_INVALID_ARG;
        if ((st = check_ffn_ws(ws, ws_bytes, T, d, n, true)) != MOE_OK) return st;
    }
    if ((st = check_arch()) != MOE_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (T == 0) {  // sums over no tokens
        cudaError_t e = cudaSuccess;
        for (void *p : {dW1, dW3, dW2})
            if (p != nullptr && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)d * n * 2, s);
        return from_cuda(e);
    }
    const FfnWs w = ffn_ws(T, d, n, true);
    return from_cuda(launch_ffn_backward(dY, X, W1, W3, W2, H, F1, F3, T, d, n,
                                         type == MOE_DTYPE_F16, at(ws, w.da1), at(ws, w.da3), dX,
                                         dW1, dW3, dW2, reinterpret_cast<float4 *>(at(ws, w.part)),
                                         reinterpret_cast<uint32_t *>(at(ws, kFfnTicketOffset)),
                                         static_cast<uint32_t *>(ws), s));
}

}  // extern "C"
