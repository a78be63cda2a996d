// Residual dropout from a counter-based generator: y = res + (keep ? x * scale : 0).
//
// Element i = row * d + column of the logical [T, d] matrix (the row strides do
// not enter) takes 16 bits of the Philox 4x32-10 block with key = seed and
// counter = (i / 8, offset) (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC11): word (i % 8) / 2, its low
// half for even i. It is kept where that number is >= thr = round(65536 p), and
// scaled by 65536 / (65536 - thr), the inverse of the probability that the draw
// really has, so that the mean stays exact although p is a multiple of 2^-16.
// The mask is never stored: the backward is the same function of dy.
//
// Bound by HBM (x, res in, y out: 6 bytes a 16-bit element) as long as the
// generator is cheap: a block of ten rounds (20 wide multiplies) serves eight
// elements, and the ten round keys are the same for all threads and come
// precomputed with the launch. 32 bits an element would double the multiplies,
// which then take as long as the memory.
//
// Elements are taken in whole generator blocks of eight. Where eight elements
// are 16-byte aligned in every tensor, a thread loads them as vectors; otherwise
// a warp takes 32 blocks = 256 elements, each lane draws one block's eight
// mask bits, and the lanes then walk the elements by one or two, neighbouring lanes on
// neighbouring elements, taking each bit from the lane that drew it. Measured with a
// residual, bf16, 8192 rows: 7168 or 7167 contiguous 54 us (6.5 TB/s), 7166 in rows of
// 7170 76 us, 7167 in rows of 7170 86 us.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct DropArgs {
    const void *x, *res;
    void *y;
    int64_t ldx, ldr, ldy;
    int64_t n;        // elements
    int64_t d;        // row length (flat: n)
    uint32_t thr;     // 0 .. 65536
    float scale;
    uint64_t offset;
    const uint64_t *offset_dev;  // added to offset, or NULL
    uint32_t k0[10], k1[10];     // round keys
};

// The keep bits of generator block g: bit j for element 8 g + j.
__device__ __forceinline__ uint32_t keep_bits(const DropArgs &a, uint64_t g, uint64_t offset) {
    uint32_t c0 = (uint32_t)g, c1 = (uint32_t)(g >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ a.k0[r];
        c2 = (uint32_t)(p >> 32) ^ c3 ^ a.k1[r];
        c1 = (uint32_t)q;
        c3 = (uint32_t)p;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t u = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
        m |= (u >= a.thr ? 1u : 0u) << j;
    }
    return m;
}

__device__ __forceinline__ float apply(const DropArgs &a, bool keep, float x, float res) {
    return keep ? fmaf(x, a.scale, res) : res;
}

// Eight elements at p (16-byte aligned) as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
    constexpr int W = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / W; ++i)
        to_f32<T, W>(reinterpret_cast<const Raw<T, W> *>(p)[i], f + i * W);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
    constexpr int W = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) reinterpret_cast<Raw<T, W> *>(p)[i] = from_f32<T, W>(f + i * W);
}

// Vector path. FLAT: one run of n elements (contiguous tensors; a last block of
// n % 8 elements goes one by one); else d % 8 == 0 and rows of d / 8 blocks.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(const DropArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t offset = a.offset + (a.offset_dev != nullptr ? *a.offset_dev : 0ull);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y);
    const int64_t blocks = (a.n + 7) / 8, step = (int64_t)gridDim.x * kThreads;
    for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < blocks; g += step) {
        int64_t ix = g * 8, ir = ix, iy = ix;
        if (!FLAT) {
            const int64_t per = a.d / 8;
            const int64_t row = blocks <= 0xffffffffll ? (int64_t)((uint32_t)g / (uint32_t)per) : g / per;
            const int64_t col = (g - row * per) * 8;
            ix = row * a.ldx + col;
            ir = row * a.ldr + col;
            iy = row * a.ldy + col;
        }
        if (FLAT && g * 8 + 8 > a.n) {
            const uint32_t m = keep_bits(a, (uint64_t)g, offset);
            for (int64_t i = g * 8; i < a.n; ++i)
                store_f32(y + i, apply(a, (m >> (i & 7)) & 1, load_f32(x + i),
                                       res != nullptr ? load_f32(res + i) : 0.f));
            continue;
        }
        float f[8], r[8];
        load8(x + ix, f);
        if (res != nullptr) {
            load8(res + ir, r);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = 0.f;
        }
        const uint32_t m = keep_bits(a, (uint64_t)g, offset);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = apply(a, (m >> j) & 1, f[j], r[j]);
        store8(y + iy, f);
    }
}

// Element path: any strides and alignment. W elements an access: 2 where every row of
// 16-bit elements starts on a word and has an even length, else 1.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) dropout_elem_kernel(const DropArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t offset = a.offset + (a.offset_dev != nullptr ? *a.offset_dev : 0ull);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y);
    constexpr int N = 8 / W;  // accesses of a lane in a run of 256 elements
    const int lane = threadIdx.x & 31;
    const int64_t runs = (a.n + 255) / 256, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t run = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); run < runs;
         run += step) {
        const int64_t i0 = run * 256;
        const int64_t row = a.n <= 0xffffff00ll ? (int64_t)((uint32_t)i0 / (uint32_t)a.d) : i0 / a.d;
        const int64_t col0 = i0 - row * a.d;
        const uint32_t m = keep_bits(a, (uint64_t)run * 32 + lane, offset);
        // elements W (32 j + lane) .. of the run: bits W lane % 8 .. of the block that lane
        // (32 j + lane) W / 8 drew
        auto bits_of = [&](int j) {
            return __shfl_sync(0xffffffffu, m, 4 * W * j + lane * W / 8) >> (lane * W & 7);
        };
        auto one = [&](Raw<T, W> qx, Raw<T, W> qr, uint32_t bits) {
            float f[W], r[W];
            to_f32<T, W>(qx, f);
            to_f32<T, W>(qr, r);
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = apply(a, (bits >> e) & 1, f[e], r[e]);
            return from_f32<T, W>(f);
        };
        Raw<T, W> fx[N], fr[N];
#pragma unroll
        for (int j = 0; j < N; ++j) fr[j] = 0;
        if (col0 + 256 <= a.d) {
            // the run lies in one row: accesses at fixed distances
            const int64_t col = col0 + lane * W;
            const Raw<T, W> *px = reinterpret_cast<const Raw<T, W> *>(x + row * a.ldx + col);
            const Raw<T, W> *pr = reinterpret_cast<const Raw<T, W> *>(res + row * a.ldr + col);
            Raw<T, W> *py = reinterpret_cast<Raw<T, W> *>(y + row * a.ldy + col);
#pragma unroll
            for (int j = 0; j < N; ++j) fx[j] = px[32 * j];
            if (res != nullptr)
#pragma unroll
                for (int j = 0; j < N; ++j) fr[j] = pr[32 * j];
#pragma unroll
            for (int j = 0; j < N; ++j) py[32 * j] = one(fx[j], fr[j], bits_of(j));
            continue;
        }
        int64_t i = i0 + lane * W, col = col0 + lane * W, at[N];
        int64_t ix = row * a.ldx + col, ir = row * a.ldr + col, iy = row * a.ldy + col;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            while (col >= a.d) {
                col -= a.d;
                ix += a.ldx - a.d;
                ir += a.ldr - a.d;
                iy += a.ldy - a.d;
            }
            at[j] = -1;
            if (i < a.n) {
                at[j] = iy;
                fx[j] = *reinterpret_cast<const Raw<T, W> *>(x + ix);
                if (res != nullptr) fr[j] = *reinterpret_cast<const Raw<T, W> *>(res + ir);
            }
            i += 32 * W;
            col += 32 * W;
            ix += 32 * W;
            ir += 32 * W;
            iy += 32 * W;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t bits = bits_of(j);
            if (at[j] >= 0) *reinterpret_cast<Raw<T, W> *>(y + at[j]) = one(fx[j], fr[j], bits);
        }
    }
}

template <typename T>
cudaError_t launch_type(DropArgs a, int64_t T_rows, cudaStream_t s) {
    const int es = sizeof(T);
    const bool has_res = a.res != nullptr;
    const uint64_t ptrs = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.res) |
                          reinterpret_cast<uintptr_t>(a.y);
    const bool flat = T_rows == 1 || (a.ldx == a.d && a.ldy == a.d && (!has_res || a.ldr == a.d));
    const uint64_t rows = (uint64_t)(a.ldx | a.ldy | (has_res ? a.ldr : 0)) * es;
    const int max_blocks = sm_count() * 8;
    if ((ptrs & 15) == 0 && (flat || (a.d % 8 == 0 && (rows & 15) == 0))) {
        const int64_t blocks = ((a.n + 7) / 8 + kThreads - 1) / kThreads;
        const dim3 grid((unsigned)std::min<int64_t>(blocks, max_blocks));
        return flat ? launch_k(dropout_vec_kernel<T, true>, grid, dim3(kThreads), 0, s, a)
                    : launch_k(dropout_vec_kernel<T, false>, grid, dim3(kThreads), 0, s, a);
    }
    const int64_t blocks = ((a.n + 255) / 256 + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid((unsigned)std::min<int64_t>(blocks, max_blocks));
    if constexpr (sizeof(T) == 2)
        if ((ptrs & 3) == 0 && a.d % 2 == 0 && (rows & 3) == 0)
            return launch_k(dropout_elem_kernel<T, 2>, grid, dim3(kThreads), 0, s, a);
    return launch_k(dropout_elem_kernel<T, 1>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_dropout(const void *x, int64_t ldx, const void *res, int64_t ldr, void *y,
                           int64_t ldy, int64_t T, int d, uint32_t thr, uint64_t seed,
                           uint64_t offset, const uint64_t *offset_dev, moe_dtype_t type,
                           cudaStream_t s) {
    DropArgs a{};
    a.x = x;
    a.res = res;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.n = T * d;
    a.d = d;
    a.thr = thr;
    a.scale = thr < 65536u ? 65536.f / (float)(65536u - thr) : 0.f;
    a.offset = offset;
    a.offset_dev = offset_dev;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int r = 0; r < 10; ++r) {
        a.k0[r] = k0;
        a.k1[r] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    switch (type) {
        case MOE_DTYPE_BF16: return launch_type<__nv_bfloat16>(a, T, s);
        case MOE_DTYPE_F16: return launch_type<__half>(a, T, s);
        default: return launch_type<float>(a, T, s);
    }
}

}  // namespace moe
