// C ABI of the sub-block operators around the layer (layer norm, residual
// dropout, dense gated feed-forward block): argument checks and launches. Errors are returned before anything
// is enqueued.
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

// The row that this thread's next layer norm withholds (moe_selftest_layernorm_withhold).
thread_local int64_t t_withheld = -1;
int64_t take_withheld() {
    const int64_t row = t_withheld;
    t_withheld = -1;
    return row;
}

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
char *at(void *ws, size_t off) { return static_cast<char *>(ws) + off; }

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
