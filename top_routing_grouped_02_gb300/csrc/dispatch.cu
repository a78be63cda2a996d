// Token rows to the rows sorted by expert and back, with the routing weights, and the
// gradients of both ways:
//   dispatch            xg[row(t,k)] = x[t]
//   sum (combine)       y[t]  = sum_k w[t,k] z[row(t,k)]  (+ residual[t]), k ascending
//     (w NULL: ones; then it is the gradient of the dispatch)
//   combine's gradient  dz[row(t,k)] = w[t,k] dy[t],  dw[t,k] = <dy[t], z[row(t,k)]>
// row(t,k) = row_of_slot[t * K + k]; a slot whose row is outside [0, rows) has none.
//
// All are bound by HBM: nothing is computed but K products an element. All go by token, so
// that a token's own row is read (or written) once and its K rows once each: the dispatch
// by sorted rows would read x K times. The slots of a token are distinct rows, so no two
// warps write the same element, and every sum has a fixed order: no atomics.
//
// A warp takes a token's elements in chunks of 32 x U vectors, with the loads of all K rows
// in flight at once. Short batches spread a token's chunks over
// more warps; the gradient, whose dot products run along the row, over the 8 warps of one
// block, which join their sums through shared memory.
// Vectors are as wide as the alignment of all operands' rows allows; the elements behind
// the last whole vector are taken one by one.
//
// Measured, 4096 x 7168 bf16, K = 8: dispatch 88 us (6.0 TB/s, nine tenths of it writes), sum
// 78 us (6.7 TB/s), with residual 86 us; gradients 155 us (6.4 TB/s). Rows of 7167, whose vectors
// are single elements: 112, 119, 131 and 281 us.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTargetWarps = 48;  // an SM

// The rows of a token's slots: every lane has all of them, -1 where a slot has none.
template <int KU>
__device__ __forceinline__ void slot_rows(const RowArgs &a, int64_t t, int lane, int64_t (&rows)[KU]) {
    int64_t mine = -1;
    if (lane < a.K) {
        mine = a.row_of_slot[t * a.K + lane];
        if (mine >= a.rows) mine = -1;
    }
#pragma unroll
    for (int k = 0; k < KU; ++k) rows[k] = __shfl_sync(0xffffffffu, (int)mine, k);
}

// Row t of a matrix of T with stride ld, as vectors of V.
template <typename T, int V>
__device__ __forceinline__ const Raw<T, V> *row_in(const void *p, int64_t ld, int64_t t) {
    return reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + t * ld);
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> *row_out(void *p, int64_t ld, int64_t t) {
    return reinterpret_cast<Raw<T, V> *>(static_cast<T *>(p) + t * ld);
}

// Vectors of a row in flight a lane: 8 of 16 or 8 bytes over all rows, more of narrower ones,
// four times as many with eight rows and twice with fewer (bf16 rows of 7167, K = 8, without
// and with: sum 177 / 119 us, gradient 416 / 281; rows of 4097, K = 2, twice and four times: sum
// 24.4 / 26.2, gradient 38.5 / 43.0; the dispatch, whose loads are one row's, four times with 2
// to 8 rows: 148 / 112, and twice with one).
template <typename T, int V, int KU>
constexpr int flight() {
    return 8 / KU * (V * (int)sizeof(T) >= 8 ? 1 : KU == 8 ? 4 : 2);
}
template <typename T, int V, int KU>
constexpr int dispatch_flight() {
    return (KU == 1 ? 8 : 4) * std::min<int>(KU == 1 ? 2 : 4, 16 / (V * (int)sizeof(T)));
}

// This warp's token and its part of the token's chunks.
struct Share {
    int64_t t;
    int part, parts;
    __device__ __forceinline__ Share(const RowArgs &a) {
        const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
        t = w / a.split;
        part = (int)(w - t * a.split);
        parts = a.split;
    }
};

template <typename T, int V, int KU>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const RowArgs a) {
    constexpr int U = dispatch_flight<T, V, KU>();
    pdl_wait();
    pdl_trigger();
    const Share s(a);
    if (s.t >= a.T) return;
    const int lane = threadIdx.x & 31, nv = a.d / V;
    int64_t rows[KU];
    slot_rows<KU>(a, s.t, lane, rows);
    const Raw<T, V> *x = row_in<T, V>(a.x, a.ldx, s.t);
    for (int c = s.part * 32 * U; c < nv; c += s.parts * 32 * U) {
        Raw<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * 32 + lane < nv) v[u] = x[c + u * 32 + lane];
#pragma unroll
        for (int k = 0; k < KU; ++k)
            if (rows[k] >= 0) {
                Raw<T, V> *to = row_out<T, V>(a.out, a.ldo, rows[k]);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * 32 + lane < nv) to[c + u * 32 + lane] = v[u];
            }
    }
    const int e = nv * V + lane;
    if (V > 1 && s.part == s.parts - 1 && e < a.d) {
        const Raw<T, 1> v = row_in<T, 1>(a.x, a.ldx, s.t)[e];
#pragma unroll
        for (int k = 0; k < KU; ++k)
            if (rows[k] >= 0) row_out<T, 1>(a.out, a.ldo, rows[k])[e] = v;
    }
}

template <typename T, int V, int KU>
__global__ void __launch_bounds__(kThreads) sum_rows_kernel(const RowArgs a) {
    constexpr int U = flight<T, V, KU>();
    pdl_wait();
    pdl_trigger();
    const Share s(a);
    if (s.t >= a.T) return;
    const int lane = threadIdx.x & 31, nv = a.d / V;
    int64_t rows[KU];
    slot_rows<KU>(a, s.t, lane, rows);
    const float wl = a.w != nullptr && lane < a.K ? a.w[s.t * a.K + lane] : 1.f;
    float w[KU];
#pragma unroll
    for (int k = 0; k < KU; ++k) w[k] = __shfl_sync(0xffffffffu, wl, k);
    // `count` vectors of `width` elements, 32 apart, from vector `first` on
    auto take = [&](auto width, auto count, int first, int end) {
        constexpr int W = width(), N = count();
        Raw<T, W> z[KU][N], r[N];
#pragma unroll
        for (int k = 0; k < KU; ++k)
            if (rows[k] >= 0) {
                const Raw<T, W> *from = row_in<T, W>(a.z, a.ldz, rows[k]);
#pragma unroll
                for (int u = 0; u < N; ++u)
                    if (first + u * 32 < end) z[k][u] = from[first + u * 32];
            }
        if (a.res != nullptr) {
            const Raw<T, W> *from = row_in<T, W>(a.res, a.ldr, s.t);
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (first + u * 32 < end) r[u] = from[first + u * 32];
        }
        Raw<T, W> *to = row_out<T, W>(a.out, a.ldo, s.t);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (first + u * 32 >= end) continue;
            float acc[W] = {}, f[W];
#pragma unroll
            for (int k = 0; k < KU; ++k)
                if (rows[k] >= 0) {
                    to_f32<T, W>(z[k][u], f);
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j] = fmaf(w[k], f[j], acc[j]);
                }
            if (a.res != nullptr) {
                to_f32<T, W>(r[u], f);
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j] += f[j];
            }
            to[first + u * 32] = from_f32<T, W>(acc);
        }
    };
    for (int c = s.part * 32 * U; c < nv; c += s.parts * 32 * U)
        take(std::integral_constant<int, V>(), std::integral_constant<int, U>(), c + lane, nv);
    if (V > 1 && s.part == s.parts - 1)
        take(std::integral_constant<int, 1>(), std::integral_constant<int, 1>(), nv * V + lane, a.d);
}

// (a.split divides the block's warps: a token's warps are of one block)
template <typename T, int V, int KU>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const RowArgs a) {
    constexpr int U = flight<T, V, KU>();
    __shared__ float part[kWarps][KU];
    pdl_wait();
    pdl_trigger();
    const Share s(a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nv = a.d / V;
    float dot[KU] = {};
    if (s.t < a.T) {
        int64_t rows[KU];
        slot_rows<KU>(a, s.t, lane, rows);
        const float wl = lane < a.K ? a.w[s.t * a.K + lane] : 0.f;
        float w[KU];
#pragma unroll
        for (int k = 0; k < KU; ++k) w[k] = __shfl_sync(0xffffffffu, wl, k);
        auto take = [&](auto width, auto count, int first, int end) {
            constexpr int W = width(), N = count();
            Raw<T, W> z[KU][N], g[N];
            const Raw<T, W> *dy = row_in<T, W>(a.x, a.ldx, s.t);
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (first + u * 32 < end) g[u] = dy[first + u * 32];
#pragma unroll
            for (int k = 0; k < KU; ++k)
                if (rows[k] >= 0) {
                    const Raw<T, W> *from = row_in<T, W>(a.z, a.ldz, rows[k]);
#pragma unroll
                    for (int u = 0; u < N; ++u)
                        if (first + u * 32 < end) z[k][u] = from[first + u * 32];
                }
#pragma unroll
            for (int u = 0; u < N; ++u) {
                if (first + u * 32 >= end) continue;
                float y[W], f[W];
                to_f32<T, W>(g[u], y);
#pragma unroll
                for (int k = 0; k < KU; ++k)
                    if (rows[k] >= 0) {
                        to_f32<T, W>(z[k][u], f);
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            dot[k] = fmaf(y[j], f[j], dot[k]);
                            f[j] = w[k] * y[j];
                        }
                        row_out<T, W>(a.out, a.ldo, rows[k])[first + u * 32] = from_f32<T, W>(f);
                    }
            }
        };
        for (int c = s.part * 32 * U; c < nv; c += s.parts * 32 * U)
            take(std::integral_constant<int, V>(), std::integral_constant<int, U>(), c + lane, nv);
        if (V > 1 && s.part == s.parts - 1)
            take(std::integral_constant<int, 1>(), std::integral_constant<int, 1>(), nv * V + lane, a.d);
    }
    float mine = 0.f;
#pragma unroll
    for (int k = 0; k < KU; ++k) {
        const float v = warp_sum(dot[k]);
        if (lane == k) mine = v;
    }
    if (s.parts > 1) {
        if (lane < KU) part[warp][lane] = mine;
        __syncthreads();
        if (s.part == 0 && lane < KU)
            for (int p = 1; p < s.parts; ++p) mine += part[warp + p][lane];
    }
    if (s.t < a.T && s.part == 0 && lane < a.K) a.dw[s.t * a.K + lane] = mine;
}

// The widest vector (in elements) at which all rows of all operands start.
int vector_width(const RowArgs &a, int esize) {
    uintptr_t bits = 0;
    auto add = [&](const void *p, int64_t ld, int64_t rows) {
        if (p == nullptr) return;
        bits |= reinterpret_cast<uintptr_t>(p);
        if (rows > 1) bits |= (uintptr_t)(ld * esize);
    };
    add(a.x, a.ldx, a.T);
    add(a.res, a.ldr, a.T);
    add(a.z, a.ldz, a.rows);
    // of tokens for the sum, of sorted rows else
    add(a.out, a.ldo, a.x == nullptr ? a.T : a.rows);
    int bytes = 16;
    while (bytes > esize && (bits & (bytes - 1)) != 0) bytes /= 2;
    while (bytes > esize && bytes / esize > a.d) bytes /= 2;
    return bytes / esize;
}

enum class Op { kDispatch, kSum, kBackward };

template <Op OP, typename T, int V, int KU>
cudaError_t launch_one(RowArgs a, cudaStream_t s) {
    constexpr int U = OP == Op::kDispatch ? dispatch_flight<T, V, KU>() : flight<T, V, KU>();
    // warps a token: enough of them to fill the device
    const int chunks = std::max(1, (a.d / V + 32 * U - 1) / (32 * U));
    const int64_t want = ((int64_t)sm_count() * kTargetWarps + a.T - 1) / a.T;
    a.split = (int)std::min<int64_t>(chunks, want);
    if (OP == Op::kBackward) {
        int p = 1;
        while (p < kWarps && p < a.split) p *= 2;
        a.split = p;
    }
    const int64_t blocks = (a.T * a.split + kWarps - 1) / kWarps;
    auto *kernel = OP == Op::kDispatch ? dispatch_kernel<T, V, KU>
                   : OP == Op::kSum    ? sum_rows_kernel<T, V, KU>
                                       : combine_backward_kernel<T, V, KU>;
    return launch_k(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
}
template <Op OP, typename T, int V>
cudaError_t launch_k_of(const RowArgs &a, cudaStream_t s) {
    if (a.K == 1) return launch_one<OP, T, V, 1>(a, s);
    if (a.K == 2) return launch_one<OP, T, V, 2>(a, s);
    if (a.K <= 4) return launch_one<OP, T, V, 4>(a, s);
    return launch_one<OP, T, V, 8>(a, s);
}
template <Op OP>
cudaError_t launch_rows(const RowArgs &a, moe_dtype_t type, cudaStream_t s) {
    const int v = vector_width(a, type == MOE_DTYPE_F32 ? 4 : 2);
    auto pick = [&](auto zero) {
        using T = decltype(zero);
        if constexpr (sizeof(T) == 2)
            if (v == 8) return launch_k_of<OP, T, 8>(a, s);
        if (v == 4) return launch_k_of<OP, T, 4>(a, s);
        if (v == 2) return launch_k_of<OP, T, 2>(a, s);
        return launch_k_of<OP, T, 1>(a, s);
    };
    if (OP == Op::kDispatch && type == MOE_DTYPE_F16) type = MOE_DTYPE_BF16;  // copied as bits
    switch (type) {
        case MOE_DTYPE_BF16: return pick(__nv_bfloat16());
        case MOE_DTYPE_F16:
            if constexpr (OP != Op::kDispatch) return pick(__half());
        default: return pick(0.f);
    }
}

}  // namespace

cudaError_t launch_dispatch(const RowArgs &a, moe_dtype_t type, cudaStream_t s) {
    return launch_rows<Op::kDispatch>(a, type, s);
}
cudaError_t launch_sum_rows(const RowArgs &a, moe_dtype_t type, cudaStream_t s) {
    return launch_rows<Op::kSum>(a, type, s);
}
cudaError_t launch_combine_backward(const RowArgs &a, moe_dtype_t type, cudaStream_t s) {
    return launch_rows<Op::kBackward>(a, type, s);
}

}  // namespace moe
