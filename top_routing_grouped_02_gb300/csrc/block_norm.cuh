// The norms around a block in one pass over the stream (block_norm.cu, its gradients in
// block_norm_backward.cu). For a row of d elements,
//   bh = b r_post,  r_post = 1 / sqrt(mean(b^2) + eps)   (1 without the post norm)
//   n  = post bh
//   y  = scale x + g n,   g = sigmoid(gate) of the row or the element, or 1
//   yh = y r_pre,   r_pre = 1 / sqrt(mean(y^2) + eps),   u = pre yh
// y is rounded for the output alone: u is that of the fp32 y. Without a block (b NULL) y = x
// and only u is written: a plain RMS norm.
#pragma once

#include "rows.cuh"

namespace moe {
namespace bn {

struct Args {
    const void *x, *b, *gate, *post, *pre;
    void *y, *u;
    float *r_post, *r_pre;
    int64_t ldx, ldb, ldg, ldy, ldu;
    int64_t T;
    int d;
    int w32;         // post, pre (and their gradients) are fp32, else x's type
    int full;        // gate is [T,d] of x's type; else one fp32 value a row, or NULL
    int post_norm, pre_norm;
    float scale, eps;
    int wpr, stages; // warps per row; ring stages per row group
    int64_t withheld;  // self-test: this row's copies are never issued (-1: none)
    // backward
    const void *dy, *du;
    void *dx, *db, *dgate;
    int64_t lddy, lddu, lddx, lddb, lddg;
    float *part;     // [blocks][2][d] partial sums (dpost, dpre), or NULL
};

// The sigmoid g of z and h = 1 - g. From t = exp(-|z|) <= 1, which neither overflows nor
// cancels: the larger of the two is 1 / (1 + t), the smaller t / (1 + t).
__device__ __forceinline__ void sigmoid(float z, float &g, float &h) {
    const float t = expf(-fabsf(z)), q = 1.f / (1.f + t), p = t * q;
    g = z < 0.f ? p : q;
    h = z < 0.f ? q : p;
}

template <typename T, int V>
__device__ __forceinline__ void load_row(const void *p, int64_t ld, int64_t row, int v, float (&f)[V]) {
    to_f32<T, V>(reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + row * ld)[v], f);
}
template <typename T, int V>
__device__ __forceinline__ void store_row(void *p, int64_t ld, int64_t row, int v, const float (&f)[V]) {
    reinterpret_cast<Raw<T, V> *>(static_cast<T *>(p) + row * ld)[v] = from_f32<T, V>(f);
}

// Sums over the warps of a row: one value each, through alternating slots, so that one
// barrier a sum is enough (who writes a slot again has passed the barrier of the sum between,
// which all others reached after they had read it).
struct GroupSum {
    float (*slots)[32];
    int w0, wpr, id, count = 0;
    __device__ __forceinline__ float operator()(float v) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        v = warp_sum(v);
        if (wpr == 1) return v;
        float *s = slots[count++ & 1];
        if (lane == 0) s[warp] = v;
        group_sync(id, wpr * 32);
        return warp_sum(lane < wpr ? s[w0 + lane] : 0.f);
    }
};

// Threads of a block without a ring, its row groups, and its grid.
constexpr int kRowThreads = 512;
struct RowShape {
    int groups, grid;
};
RowShape row_shape(Args &a, int per_thread);

}  // namespace bn
}  // namespace moe
