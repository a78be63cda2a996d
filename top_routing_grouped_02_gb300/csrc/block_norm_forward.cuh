// The norms around a block (block_norm.cuh), forward, for one element type: y and u from x, b and the gate.
//
// Bound by HBM: x, b and the gate are read once, y and u written once. A group of warps
// takes a row; r_post needs the whole row of b before y can be formed, and r_pre the whole
// row of y before u can: two sums over the group, with y in registers from the first to the
// end.
//
// Measured, calls back to back: 8192 x 7168 bf16 with a full gate 103 us (5.7 TB/s), 4096 x 4096
// bf16 with a row's gate 25 us (5.3 TB/s), 8192 x 4097 fp32 89 us (6.0 TB/s); rows of 7167 bf16
// 113 us, of 7168 with inputs that start elsewhere than outputs 153 us.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace bn {
namespace {

// Rows that no ring holds, straight from global memory (b is read twice, the second time from
// L1). A thread has NV vectors of V elements of a row, a group of warps apart: 16 elements.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) forward_rows_kernel(const Args a) {
    __shared__ float slots[2][32];
    pdl_wait();
    pdl_trigger();
    const int tpr = a.wpr * 32, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int groups = blockDim.x / tpr, nvec = a.d / V;
    const float inv_d = 1.f / (float)a.d;
    GroupSum sum{slots, group * a.wpr, a.wpr, 1 + group};
    for (int64_t row = (int64_t)blockIdx.x * groups + group; row < a.T; row += (int64_t)gridDim.x * groups) {
        float f[V], y[NV][V], r_post = 1.f, g = 1.f, h;
        if (a.gate != nullptr && !a.full) sigmoid(static_cast<const float *>(a.gate)[row], g, h);
        if (a.post_norm) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tpr + t;
                if (v >= nvec) continue;
                load_row<T, V>(a.b, a.ldb, row, v, f);
#pragma unroll
                for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
            }
            r_post = __frsqrt_rn(sum(s) * inv_d + a.eps);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t;
            if (v >= nvec) continue;
            load_row<T, V>(a.x, a.ldx, row, v, y[i]);
            if (a.b != nullptr) {
                float z[V];
                load_row<T, V>(a.b, a.ldb, row, v, f);
                if (a.full) load_row<T, V>(a.gate, a.ldg, row, v, z);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float n = f[j] * r_post * load_w<T>(a.post, a.w32, v * V + j, 1.f);
                    if (a.full) sigmoid(z[j], g, h);
                    y[i][j] = fmaf(a.scale, y[i][j], g * n);
                }
                store_row<T, V>(a.y, a.ldy, row, v, y[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(y[i][j], y[i][j], s);
        }
        if (t == 0 && a.post_norm && a.r_post != nullptr) a.r_post[row] = r_post;
        if (!a.pre_norm) continue;
        const float r_pre = __frsqrt_rn(sum(s) * inv_d + a.eps);
        if (t == 0 && a.r_pre != nullptr) a.r_pre[row] = r_pre;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t;
            if (v >= nvec) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = y[i][j] * r_pre * load_w<T>(a.pre, a.w32, v * V + j, 1.f);
            store_row<T, V>(a.u, a.ldu, row, v, f);
        }
    }
}

template <typename T, int V, int NV>
cudaError_t forward_rows(Args a, cudaStream_t s) {
    const RowShape r = row_shape(a, V * NV);
    return launch_k(forward_rows_kernel<T, V, NV>, dim3(r.grid), dim3(r.groups * a.wpr * 32), 0, s, a);
}

// Rows through a ring. MODE: 0 x alone, 1 x and b (a gate is the row's), 2 x, b and the gate.
// The arithmetic is packed.
constexpr int kFwdThreads = 896, kFwdWideThreads = 640;  // most of a block; with 32 elements a thread
template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW>
__global__ void __launch_bounds__(V * NV == 32 ? kFwdWideThreads : kFwdThreads, 1) forward_ring_kernel(const Args a) {
    extern __shared__ __align__(128) uint8_t ring_sh[];
    RingCtl *ctl = reinterpret_cast<RingCtl *>(ring_sh);
    using Wt = Weights<T, V, SHIFT, RAW>;
    constexpr int P2 = V / 2, K = MODE + 1 + (MODE == 1);  // (a stage's tensors, and a row's gate)
    const int tpr = a.wpr * 32, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int groups = blockDim.x / tpr, S = a.stages;
    const uint32_t row_bytes = ring_row_bytes<T, SHIFT>(a.d);
    const uint32_t stage_bytes = (MODE + 1) * row_bytes, w_bytes = Wt::bytes(a.d);
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    if (SHIFT) row = blockIdx.x % kPhases + (int64_t)kPhases * (blockIdx.x / kPhases * groups + group);
    // (the rows of a block start at the same place: its first row's, there or not)
    const Part<T, V, SHIFT> part(tpr, t, a.d, static_cast<T *>(MODE > 0 ? a.y : a.u) + blockIdx.x % kPhases * (MODE > 0 ? a.ldy : a.ldu));
    uint8_t *post = ring_sh + kRingCtl, *pre = post + (MODE > 0 ? w_bytes : 0);
    uint8_t *ring = pre + w_bytes + (size_t)group * a.group_bytes;
    const uint32_t bar0 = ptx::smem_addr(&ctl->full[group][0]);
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(bar0 + 8 * s, K);
        ptx::fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    // row r of tensor k (x, b, gate) into stage s: a thread each
    auto fetch = [&](int64_t r, int s, int k) {
        if (r == a.withheld) return;
        if (MODE == 1 && k == 2) {
            fetch_scalars(ctl->scalars[group][s], nullptr, nullptr, static_cast<const float *>(a.gate), r, bar0 + 8 * s);
            return;
        }
        fetch_row<T, SHIFT>(ring + (size_t)s * stage_bytes + (size_t)k * row_bytes, k == 0 ? a.x : k == 1 ? a.b : a.gate,
                            k == 0 ? a.ldx : k == 1 ? a.ldb : a.ldg, r, a.T, a.d, bar0 + 8 * s);
    };
    __syncwarp();
    if (t < S * K && row + t / K * stride < a.T) fetch(row + t / K * stride, t / K, t % K);
    if (MODE > 0) Wt::fill(post, a.post, a.w32, part);
    Wt::fill(pre, a.pre, a.w32, part);
    __syncthreads();

    auto off = [&](const void *p, int64_t ld) { return part.off(static_cast<const T *>(p) + blockIdx.x % kPhases * ld); };
    const int ox = off(a.x, a.ldx), ob = MODE > 0 ? off(a.b, a.ldb) : 0, oz = MODE > 1 ? off(a.gate, a.ldg) : 0;
    const int oy = 0, ou = MODE > 0 ? off(a.u, a.ldu) : 0;
    const float inv_d = 1.f / (float)a.d;
    GroupSum sum{ctl->slots, group * a.wpr, a.wpr, 1 + group};
    int s = 0;
    uint32_t ph = 0;
    bool alive = true;
    for (; row < a.T; row += stride) {
        alive = alive && ring_wait(bar0, S, s, ph, t < K);
        float g_row = 1.f, h_row;
        if (MODE == 1 && a.gate != nullptr) sigmoid(ctl->scalars[group][s][2], g_row, h_row);
        const uint8_t *stage = ring + (size_t)s * stage_bytes;
        const uint8_t *px = stage + image_at<T, SHIFT>(a.x, a.ldx, row);
        const uint8_t *pb = stage + row_bytes + (MODE > 0 ? image_at<T, SHIFT>(a.b, a.ldb, row) : 0);
        const uint8_t *pz = stage + 2 * row_bytes + (MODE > 1 ? image_at<T, SHIFT>(a.gate, a.ldg, row) : 0);
        float r_post = 1.f;
        if (MODE > 0 && a.post_norm) {
            f32x2 q = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!part.has(i)) continue;
                f32x2 b[P2];
                part.load(pb, ob, i, b);
#pragma unroll
                for (int j = 0; j < P2; ++j) q = fma2(b[j], b[j], q);
            }
            r_post = __frsqrt_rn(sum(pair_sum(q)) * inv_d + a.eps);
            if (t == 0 && a.r_post != nullptr) a.r_post[row] = alive ? r_post : NAN;
        }
        f32x2 y[NV][P2], q = alive ? 0 : both(NAN);
        // (a row that did not come: NaN)
        const f32x2 scale = both(alive ? a.scale : NAN), rp = both(r_post * g_row);
        T *yrow = static_cast<T *>(a.y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!part.has(i)) continue;
            part.load(px, ox, i, y[i]);
            if (MODE > 0) {
                f32x2 b[P2], w[P2];
                part.load(pb, ob, i, b);
                Wt::load(part, post, i, w);
                if (MODE == 2) {
                    f32x2 z[P2], g, h;
                    part.load(pz, oz, i, z);
#pragma unroll
                    for (int j = 0; j < P2; ++j) {
                        sigmoid2<T, false>(z[j], g, h);
                        w[j] = mul2(w[j], g);
                    }
                }
#pragma unroll
                for (int j = 0; j < P2; ++j) y[i][j] = fma2(scale, y[i][j], mul2(mul2(b[j], rp), w[j]));
                part.store(yrow, oy, i, y[i]);
            }
#pragma unroll
            for (int j = 0; j < P2; ++j) q = fma2(y[i][j], y[i][j], q);
        }
        float ss = 0.f;
        if (a.pre_norm) ss = sum(pair_sum(q));
        else if (a.wpr > 1) group_sync(1 + group, tpr);
        if (a.wpr == 1) __syncwarp();
        // every thread of the group is done with the stage
        if (t < K && alive && row + S * stride < a.T) fetch(row + S * stride, s, t);
        if (a.pre_norm) {
            const float r_pre = __frsqrt_rn(ss * inv_d + a.eps);
            if (t == 0 && a.r_pre != nullptr) a.r_pre[row] = r_pre;
            const f32x2 rq = both(r_pre);
            T *urow = static_cast<T *>(a.u) + row * a.ldu;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!part.has(i)) continue;
                f32x2 w[P2];
                Wt::load(part, pre, i, w);
#pragma unroll
                for (int j = 0; j < P2; ++j) w[j] = mul2(mul2(y[i][j], rq), w[j]);
                part.store(urow, ou, i, w);
            }
        }
        if (++s == S) {
            s = 0;
            ph ^= 1;
        }
    }
}

template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW>
bool forward_shape(Args &a, int *groups, size_t *smem) {
    const size_t stage = (MODE + 1) * ring_row_bytes<T, SHIFT>(a.d);
    const size_t fixed = kRingCtl + (MODE > 0 ? 2 : 1) * Weights<T, V, SHIFT, RAW>::bytes(a.d);
    if (!shape_of(a, ring_cols<V, SHIFT>(a.d), V * NV, V * NV == 32 ? kFwdWideThreads : kFwdThreads, sm_count(),
                    fixed, stage, stage, groups)) return false;
    *smem = fixed + (size_t)*groups * a.group_bytes;
    return true;
}
template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW>
cudaError_t forward_launch(const Args &a, int groups, size_t smem, cudaStream_t s) {
    const auto kernel = forward_ring_kernel<T, V, NV, MODE, SHIFT, RAW>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)kRingSmem);
    if (e != cudaSuccess) return e;
    return launch_k(kernel, dim3(ring_grid<SHIFT>(a.T, groups, sm_count())), dim3(groups * a.wpr * 32), smem, s, a);
}
// 16-bit weights as they are where their planes leave room for fewer rows at a time (8192 x 7168
// bf16 with a full gate, 113 / 103 us; 8192 x 2048 fp16, where both leave the same, 31.8 with planes, 32.2).
template <typename T, int NV, int MODE, int SHIFT>
cudaError_t forward_ring(const Args &a, bool *fits, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    Args planes = a;
    int groups = 0;
    size_t smem = 0;
    *fits = forward_shape<T, V, NV, MODE, SHIFT, false>(planes, &groups, &smem);
    if constexpr (sizeof(T) == 2) {
        Args raw = a;
        int more = 0;
        size_t less = 0;
        if (!a.w32 && forward_shape<T, V, NV, MODE, SHIFT, true>(raw, &more, &less) &&
            (!*fits || rows_ahead(raw, more) > rows_ahead(planes, groups))) {
            *fits = true;
            return forward_launch<T, V, NV, MODE, SHIFT, true>(raw, more, less, s);
        }
    }
    return *fits ? forward_launch<T, V, NV, MODE, SHIFT, false>(planes, groups, smem, s) : cudaSuccess;
}
// 16 elements a thread, or 32 (16-bit types): of long rows that start anywhere (8192 x 7167 bf16 with a
// full gate 149 / 113 us, 8192 x 4097 with a row's 61 / 54), and of rows that 16 do not reach over.
// Where inputs start elsewhere than outputs behind a block, 16 as long as a block holds two rows so
// (8192 x 2048 with a row's gate 43.7 / 43.2, 8192 x 4096 70 / 77, with a full one 76 / 91, 4096 x 6144
// 56 / 67 and 61 / 69; 4096 x 7168, one row, 87 / 71 and 93 / 85, 8192 x 7168 179 / 153; the norm
// alone, 8192 x 2560, 25.6 / 22.5, 4096 x 7168 42.5 / 30.1). Aligned rows: 8192 x 2048 28.5 / 31.7 us,
// 4096 x 4096 28.5 / 32.3, 8192 x 6144 with a row's gate 66 / 74 (4096 x 4096, 25.5 / 24.5).
template <typename T, int MODE, int SHIFT>
cudaError_t forward_length(const Args &a, bool *fits, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool two_rows = SHIFT == 2 && MODE > 0 && 2 * ring_cols<V, SHIFT>(a.d) <= kFwdThreads * 16;
    if (sizeof(T) == 4 || SHIFT == 0 || a.d < 2048 || two_rows) {
        const cudaError_t e = forward_ring<T, 16 / V, MODE, SHIFT>(a, fits, s);
        if (sizeof(T) == 4 || e != cudaSuccess || *fits) return e;
    }
    if constexpr (sizeof(T) == 2) return forward_ring<T, 32 / V, MODE, SHIFT>(a, fits, s);
    return cudaSuccess;
}
template <typename T, int SHIFT>
cudaError_t forward_rings(const Args &a, bool *fits, cudaStream_t s) {
    return a.b == nullptr ? forward_length<T, 0, SHIFT>(a, fits, s)
           : !a.full      ? forward_length<T, 1, SHIFT>(a, fits, s)
                          : forward_length<T, 2, SHIFT>(a, fits, s);
}

}  // namespace

template <typename T>
cudaError_t forward_type(const Args &a, int shift, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    bool fits = false;
    const cudaError_t e = shift == 0   ? forward_rings<T, 0>(a, &fits, s)
                          : shift == 1 ? forward_rings<T, 1>(a, &fits, s)
                                       : forward_rings<T, 2>(a, &fits, s);
    if (e != cudaSuccess || fits) return e;
    return shift == 0 ? forward_rows<T, W, 16 / W>(a, s) : forward_rows<T, 1, 16>(a, s);
}

}  // namespace bn
}  // namespace moe
