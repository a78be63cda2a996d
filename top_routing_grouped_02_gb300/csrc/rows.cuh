// Shared by the kernels that take rows by groups of warps (layer norm, block norm): sums over
// warps, weights, rings of rows in shared memory and the alignment of operands.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Element c of a weight vector of T or (w32) fp32, `none` without one.
template <typename T>
__device__ __forceinline__ float load_w(const void *w, int w32, int c, float none) {
    if (w == nullptr) return none;
    return w32 ? static_cast<const float *>(w)[c] : load_f32(static_cast<const T *>(w) + c);
}

// ---- rings of rows, filled by bulk copies

// The shape of a block with one ring for each of its row groups, one block per SM.
struct Ring {
    int wpr, groups, stages;  // warps a row; row groups; stages of each
};
struct RingNeeds {
    int64_t T;
    int cols, per_thread;  // columns that a row's vectors may reach over; elements a thread
    int max_threads, max_groups, max_stages, sms;
    size_t fixed, extra;   // bytes a block; bytes a group beside its ring
    size_t stage, least;   // bytes a stage; of a group's ring at least (one stage or more)
};
constexpr size_t kRingSmem = 224 * 1024;
// As many groups as have `least` each, at most T / SMs rounded up, so that few rows spread over the
// SMs; then as many stages as there is room for. False where one group does not fit.
inline bool ring_shape(const RingNeeds &n, Ring *r) {
    if (n.cols > n.max_threads * n.per_thread) return false;
    r->wpr = (n.cols + n.per_thread * 32 - 1) / (n.per_thread * 32);
    // (named barriers: 15)
    int g = std::min(std::max(1, n.max_threads / (32 * r->wpr)), r->wpr > 1 ? 15 : n.max_groups);
    g = (int)std::min<int64_t>(g, std::max<int64_t>(1, (n.T + n.sms - 1) / n.sms));
    while (g > 1 && n.fixed + g * (n.extra + n.least) > kRingSmem) --g;
    if (n.fixed + g * (n.extra + n.least) > kRingSmem) return false;
    r->groups = g;
    r->stages = (int)std::min<size_t>(((kRingSmem - n.fixed) / g - n.extra) / n.stage, n.max_stages);
    return true;
}

constexpr uint64_t kWaitLimitNs = 1000000000ull;

// Waits for stage s. A copy that has not arrived after about a second never will (it was
// issued by this block: the device has stopped). Then false, and the caller's group gives
// up: it issues no further copies, its rows' results and the block's sums become NaN. Copies
// in flight land before the block leaves, as far as another limit allows (drain: the
// threads that issue copies wait for them).
static __device__ __noinline__ bool ring_wait_long(uint32_t bar0, int stages, int s, uint32_t parity, bool drain) {
    uint64_t t0 = ptx::globaltimer_ns();
    for (;;) {
        // the clock first: a block that was held up for longer looks once more
        const bool late = ptx::globaltimer_ns() - t0 > kWaitLimitNs;
        if (ptx::mbar_try_wait(bar0 + 8 * s, parity)) return true;
        if (late) break;
    }
    t0 = ptx::globaltimer_ns();
    for (int k = 0; drain && k < stages; ++k) {
        const int at = s + k < stages ? s + k : s + k - stages;
        while (!ptx::mbar_try_wait(bar0 + 8 * at, s + k < stages ? parity : parity ^ 1))
            if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
    return false;
}
__device__ __forceinline__ bool ring_wait(uint32_t bar0, int stages, int s, uint32_t parity, bool drain) {
    return ptx::mbar_try_wait(bar0 + 8 * s, parity) || ring_wait_long(bar0, stages, s, parity, drain);
}

// Weights of vector v from their planes.
template <int V>
__device__ __forceinline__ void plane_pairs(const float *planes, int nvec, int v, f32x2 (&g)[V / 2]) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(planes + (h * nvec + v) * 4);
        g[2 * h] = q.x;
        g[2 * h + 1] = q.y;
    }
}
template <typename T, int V>
__device__ __forceinline__ void fill_planes(float *planes, const void *w, int w32, int d, float none) {
    const int nvec = (d + V - 1) / V;
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = v * V + j < d ? load_w<T>(w, w32, v * V + j, none) : 0.f;
#pragma unroll
        for (int h = 0; h < V / 4; ++h)
            *reinterpret_cast<float4 *>(planes + (h * nvec + v) * 4) =
                make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    }
}

// A block's partial sums of two weight gradients: each group puts its own into its ring (as
// planes, [2][d rounded up to V]), and the block adds the groups' in order, four columns a
// thread. (One group after the other through one copy took 3.5 us for 4 groups of d =
// 4096.)
template <int V, int NV>
__device__ __forceinline__ void store_partials(float *parts, int d, int groups, int group, int tpr,
                                               int t, const bool (&ok)[NV],
                                               const f32x2 (&dg)[NV][V / 2],
                                               const f32x2 (&db)[NV][V / 2], uint8_t *rings,
                                               size_t ring_bytes, bool gave_up) {
    float *part = parts + (int64_t)blockIdx.x * 2 * d;
    const int nvec = (d + V - 1) / V;
    constexpr int H = V / 4;
    // every thread is done with the last rows
    const bool lost = __syncthreads_or(gave_up);
    float4 *mine = reinterpret_cast<float4 *>(rings + group * ring_bytes);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (ok[i])
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const f32x2 *p = m == 0 ? &dg[i][2 * h] : &db[i][2 * h];
                    float4 q;
                    unpair(p[0], q.x, q.y);
                    unpair(p[1], q.z, q.w);
                    mine[(m * H + h) * nvec + i * tpr + t] = q;
                }
    __syncthreads();
    const int quads = nvec * H;  // of one array
    for (int c = threadIdx.x; c < 2 * quads; c += blockDim.x) {
        const int m = c >= quads, e = c - m * quads, v = e / H, h = e % H;
        if (4 * e >= d) continue;  // the last vector may reach past the row
        const uint8_t *at = rings + (size_t)((m * H + h) * nvec + v) * sizeof(float4);
        float4 x = *reinterpret_cast<const float4 *>(at);
        for (int k = 1; k < groups; ++k) {
            const float4 q = *reinterpret_cast<const float4 *>(at + k * ring_bytes);
            x.x += q.x;
            x.y += q.y;
            x.z += q.z;
            x.w += q.w;
        }
        if (lost) x.x = x.y = x.z = x.w = NAN;
        float *out = part + (int64_t)m * d + 4 * e;
        if ((d & 3) == 0) {
            *reinterpret_cast<float4 *>(out) = x;
        } else {
            const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * e + j < d) out[j] = f[j];
        }
    }
}

// ---- rows that start anywhere: images of their 16-byte blocks

// Bytes of the image of a row: its blocks, wherever it starts, and one more that the
// last vector's shift reads.
__host__ __device__ constexpr uint32_t image_bytes(int d, int esize) {
    return ((uint32_t)d * esize + 15) / 16 * 16 + 32;  // (d: of a row that fits the ring)
}
// One thread: the blocks of row r of a [T, d] tensor into img, announced on bar
// (which the caller arrives on, with the bytes returned). Elements in blocks that reach
// out of the tensor are copied one by one.
template <typename T>
__device__ __forceinline__ uint32_t fetch_image(uint8_t *img, const T *base, int64_t ld, int64_t r,
                                                int64_t rows, int d, uint32_t bar) {
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(base);
    const uintptr_t b1 = reinterpret_cast<uintptr_t>(base + (rows - 1) * ld + d);
    const T *row = base + r * ld;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row), end = reinterpret_cast<uintptr_t>(row + d);
    const uintptr_t origin = at & ~(uintptr_t)15;
    uintptr_t lo = origin, hi = (end + 15) & ~(uintptr_t)15;
    if (lo < b0) lo += 16;
    if (hi > b1) hi -= 16;
    uint32_t bytes = 0;
    if (hi > lo) {
        bytes = (uint32_t)(hi - lo);
        ptx::bulk_load(ptx::smem_addr(img + (lo - origin)), reinterpret_cast<const void *>(lo), bytes, bar);
    } else {
        lo = hi = end;  // no whole block: every element by itself
    }
    T *to = reinterpret_cast<T *>(img + (at - origin));
    for (const T *p = row; reinterpret_cast<uintptr_t>(p) < lo; ++p) to[p - row] = *p;
    if (hi < end)
        for (const T *p = reinterpret_cast<const T *>(hi); p < row + d; ++p) to[p - row] = *p;
    return bytes;
}
// The 16 bytes of vector v of a row whose image starts `shift` bytes into img.
template <typename T>
__device__ __forceinline__ uint4 image_vec(const uint8_t *img, int v, uint32_t shift) {
    const uint4 a = reinterpret_cast<const uint4 *>(img)[v], b = reinterpret_cast<const uint4 *>(img)[v + 1];
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x;
    if (shift & 8) {
        w0 = a.z;
        w1 = a.w;
        w2 = b.x;
        w3 = b.y;
        w4 = b.z;
    }
    if (shift & 4) {
        w0 = w1;
        w1 = w2;
        w2 = w3;
        w3 = w4;
        w4 = shift & 8 ? b.w : b.y;
    }
    if (sizeof(T) == 4) return make_uint4(w0, w1, w2, w3);
    const uint32_t bits = (shift & 2) * 8;
    return make_uint4(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits),
                      __funnelshift_r(w2, w3, bits), __funnelshift_r(w3, w4, bits));
}

// What all rows of the operands are aligned to.
struct Align {
    uint64_t bits = 0;
    void add(const void *p, int64_t ld, int d, int esize, int64_t T) {
        if (p == nullptr) return;
        bits |= reinterpret_cast<uintptr_t>(p) | (uint64_t)d * esize;
        if (T > 1) bits |= (uint64_t)ld * esize;
    }
    bool fits(int bytes) const { return (bits & (bytes - 1)) == 0; }
};

}  // namespace moe
