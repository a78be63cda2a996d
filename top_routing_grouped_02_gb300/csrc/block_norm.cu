// The norms around a block (block_norm.cuh), forward: y and u from x, b and the gate.
//
// Bound by HBM: x, b and the gate are read once, y and u written once. A group of warps
// takes a row; r_post needs the whole row of b before y can be formed, and r_pre the whole
// row of y before u can: two sums over the group, with y in registers from the first to the
// end.
#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace bn {
namespace {

// Rows of any alignment, straight from global memory (b is read twice, the second time from
// L1). A thread has NV vectors of V elements of a row, a group of warps apart.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(V * NV >= 16 ? 1024 : kRowThreads) forward_rows_kernel(const Args a) {
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
        if (t == 0 && a.r_post != nullptr) a.r_post[row] = r_post;
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

template <typename T>
cudaError_t forward_type(const Args &a, const Align &al, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if (al.fits(16)) return forward_rows<T, W, 16 / W>(a, s);
    if (a.d <= 32) return forward_rows<T, 1, 1>(a, s);
    if (a.d <= 4 * kRowThreads) return forward_rows<T, 1, 4>(a, s);
    return forward_rows<T, 1, 16>(a, s);
}

}  // namespace

RowShape row_shape(Args &a, int per_thread) {
    a.wpr = (a.d + per_thread * 32 - 1) / (per_thread * 32);
    RowShape r;
    r.groups = std::max(1, std::min(kRowThreads / (32 * a.wpr), 15));
    // few rows spread over the SMs
    r.groups = (int)std::min<int64_t>(r.groups, std::max<int64_t>(1, (a.T + sm_count() - 1) / sm_count()));
    r.grid = (int)std::min<int64_t>((a.T + r.groups - 1) / r.groups, 4 * sm_count());
    return r;
}

}  // namespace bn

using namespace bn;

cudaError_t launch_block_norm_forward(const BlockNormCall &c, int64_t withheld, cudaStream_t s) {
    Args a{};
    Align al;
    const int es = c.type == MOE_DTYPE_F32 ? 4 : 2;
    auto in = [&](const Matrix &m) {
        al.add(m.p, m.ld, c.d, es, c.T);
        return m.p;
    };
    a.x = in(c.x);
    a.ldx = c.x.ld;
    a.b = in(c.b);
    a.ldb = c.b.ld;
    a.full = c.gate.p != nullptr && c.gate_rows;
    a.gate = a.full ? in(c.gate) : c.gate.p;
    a.ldg = c.gate.ld;
    a.y = const_cast<void *>(in(c.y));
    a.ldy = c.y.ld;
    a.u = const_cast<void *>(in(c.u));
    a.ldu = c.u.ld;
    a.post = c.post;
    a.pre = c.pre;
    a.r_post = c.r_post;
    a.r_pre = c.r_pre;
    a.T = c.T;
    a.d = c.d;
    a.w32 = c.w32;
    a.post_norm = c.post_norm;
    a.pre_norm = c.pre_norm;
    a.scale = c.scale;
    a.eps = c.eps;
    a.withheld = withheld;
    switch (c.type) {
        case MOE_DTYPE_BF16: return forward_type<__nv_bfloat16>(a, al, s);
        case MOE_DTYPE_F16: return forward_type<__half>(a, al, s);
        default: return forward_type<float>(a, al, s);
    }
}

}  // namespace moe
