// Shared by the kernels that take rows by groups of warps (layer norm, block norm): sums over
// warps, weights, rings of rows in shared memory and the alignment of operands.
#pragma once

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
