// The norms around a block (block_norm.cuh), gradients: with e = pre du,
//   dY   = dy + r_pre (e - yh mean(e yh))          the whole gradient of y
//   f    = g dY post                               the gradient of bh
//   dx   = scale dY,   db = r_post (f - bh mean(f bh))
//   dgate = dY n g (1 - g) = f bh (1 - g), of a row's gate summed over the row
//   dpost = sum over rows of g dY bh,   dpre = sum over rows of du yh
// y is formed again from x, b and the gate, in fp32, as in the forward (reading the rounded y
// instead would cost as much and lose the rounded bits).
//
// Bound by HBM: x, b, the gate, dy and du are read once, dx, db and dgate written once. Two
// sums over a row: e yh before dY, f bh before db (a row's dgate is (1 - g) times the
// second). Each thread owns its columns and sums dpost and dpre over its group's rows in
// registers; a block's groups are added in order through shared memory, the blocks' partial
// rows by a second kernel, in order: no atomics, the result does not depend on timing.
#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace bn {
namespace {

// Rows of any alignment, straight from global memory. What fits (KEEP) stays in registers
// from pass to pass; else each pass forms it again, from L1 or L2. All results are written
// by the last pass, after the thread's last read, so that they may replace inputs.
template <typename T, int V, int NV, bool KEEP>
__global__ void __launch_bounds__(V * NV >= 16 ? 1024 : kRowThreads)
backward_rows_kernel(const Args a) {
    extern __shared__ float sums[];  // [groups][2][d]
    __shared__ float slots[2][32];
    pdl_wait();
    pdl_trigger();
    const int tpr = a.wpr * 32, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int groups = blockDim.x / tpr, nvec = a.d / V;
    const float inv_d = 1.f / (float)a.d;
    GroupSum sum{slots, group * a.wpr, a.wpr, 1 + group};
    float dpost[NV][V], dpre[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dpost[i][j] = dpre[i][j] = 0.f;
    for (int64_t row = (int64_t)blockIdx.x * groups + group; row < a.T; row += (int64_t)gridDim.x * groups) {
        const float r_post = a.post_norm ? a.r_post[row] : 1.f, r_pre = a.pre_norm ? a.r_pre[row] : 0.f;
        float g_row = 1.f, h_row = 0.f;
        if (a.gate != nullptr && !a.full) sigmoid(static_cast<const float *>(a.gate)[row], g_row, h_row);
        constexpr int K = KEEP ? NV : 1;
        // of a vector: yh, bh, g and 1 - g, du and (the gradient of y) dy
        float yh[K][V], bh[K][V], g[K][V], h[K][V], du[K][V], dy[K][V];
        auto form = [&](int i, int v) {
            const int k = KEEP ? i : 0;
            float x[V], z[V];
            load_row<T, V>(a.x, a.ldx, row, v, x);
            if (a.b != nullptr) load_row<T, V>(a.b, a.ldb, row, v, bh[k]);
            if (a.full) load_row<T, V>(a.gate, a.ldg, row, v, z);
            if (a.pre_norm) load_row<T, V>(a.du, a.lddu, row, v, du[k]);
            if (a.dy != nullptr) load_row<T, V>(a.dy, a.lddy, row, v, dy[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[k][j] = g_row;
                h[k][j] = h_row;
                if (a.full) sigmoid(z[j], g[k][j], h[k][j]);
                float y = x[j];
                if (a.b != nullptr) {
                    bh[k][j] *= r_post;
                    y = fmaf(a.scale, y, g[k][j] * (bh[k][j] * load_w<T>(a.post, a.w32, v * V + j, 1.f)));
                } else {
                    bh[k][j] = 0.f;
                }
                yh[k][j] = y * r_pre;
                if (!a.pre_norm) du[k][j] = 0.f;
                if (a.dy == nullptr) dy[k][j] = 0.f;
            }
        };
        auto weight = [&](const void *w, int v, int j) { return load_w<T>(w, a.w32, v * V + j, 1.f); };
        float s = 0.f;
        if (KEEP || a.pre_norm) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tpr + t, k = KEEP ? i : 0;
                if (v >= nvec) continue;
                form(i, v);
#pragma unroll
                for (int j = 0; j < V; ++j) s = fmaf(du[k][j] * weight(a.pre, v, j), yh[k][j], s);
            }
        }
        const float c1 = a.pre_norm ? sum(s) * inv_d : 0.f;
        // dY of element j of vector v
        auto grad_y = [&](int k, int v, int j) {
            return fmaf(r_pre, fmaf(-c1, yh[k][j], du[k][j] * weight(a.pre, v, j)), dy[k][j]);
        };
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t, k = KEEP ? i : 0;
            if (v >= nvec) continue;
            if (!KEEP) form(i, v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gd = g[k][j] * grad_y(k, v, j) * bh[k][j];
                dpost[i][j] += gd;
                dpre[i][j] = fmaf(du[k][j], yh[k][j], dpre[i][j]);
                s = fmaf(gd, weight(a.post, v, j), s);
            }
        }
        if (a.b != nullptr) s = sum(s);
        const float c2 = a.post_norm ? s * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t, k = KEEP ? i : 0;
            if (v >= nvec) continue;
            if (!KEEP) form(i, v);
            float dx[V], db[V], dz[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gy = grad_y(k, v, j), f = g[k][j] * gy * weight(a.post, v, j);
                dx[j] = a.b != nullptr ? a.scale * gy : gy;
                dz[j] = f * bh[k][j] * h[k][j];
                db[j] = r_post * fmaf(-c2, bh[k][j], f);
            }
            store_row<T, V>(a.dx, a.lddx, row, v, dx);
            if (a.b != nullptr) store_row<T, V>(a.db, a.lddb, row, v, db);
            if (a.full) store_row<T, V>(a.dgate, a.lddg, row, v, dz);
        }
        if (t == 0 && a.gate != nullptr && !a.full) static_cast<float *>(a.dgate)[row] = h_row * s;
    }
    if (a.part == nullptr) return;
    // the groups' sums in order
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * tpr + t;
        if (v >= nvec) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sums[(size_t)(2 * group) * a.d + v * V + j] = dpost[i][j];
            sums[(size_t)(2 * group + 1) * a.d + v * V + j] = dpre[i][j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) {
        float s = sums[c];
        for (int k = 1; k < groups; ++k) s += sums[(size_t)2 * k * a.d + c];
        a.part[(size_t)blockIdx.x * 2 * a.d + c] = s;
    }
}

template <typename T, int V, int NV, bool KEEP>
cudaError_t backward_rows(Args a, int *P, cudaStream_t s) {
    RowShape r = row_shape(a, V * NV);
    r.grid = std::min(r.grid, kLnPartials);
    *P = r.grid;
    const size_t smem = a.part != nullptr ? (size_t)r.groups * 2 * a.d * sizeof(float) : 0;
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(backward_rows_kernel<T, V, NV, KEEP>), (int)(2 * kBlockNormMaxWidth * sizeof(float)));
    if (e != cudaSuccess) return e;
    return launch_k(backward_rows_kernel<T, V, NV, KEEP>, dim3(r.grid), dim3(r.groups * a.wpr * 32), smem, s, a);
}

template <typename T>
cudaError_t backward_type(const Args &a, const Align &al, moe_dtype_t type, void *dpost, void *dpre,
                          cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    int P = 0;
    cudaError_t e;
    if (al.fits(16)) e = backward_rows<T, W, 16 / W, false>(a, &P, s);
    else if (a.d <= 32) e = backward_rows<T, 1, 1, true>(a, &P, s);
    else if (a.d <= 4 * kRowThreads) e = backward_rows<T, 1, 4, true>(a, &P, s);
    else e = backward_rows<T, 1, 16, false>(a, &P, s);
    if (e != cudaSuccess || a.part == nullptr) return e;
    return launch_weight_reduce(a.part, P, a.d, a.w32 ? MOE_DTYPE_F32 : type, dpost, dpre, s);
}

}  // namespace
}  // namespace bn

using namespace bn;

cudaError_t launch_block_norm_backward(const BlockNormCall &c, int64_t withheld, cudaStream_t s) {
    Args a{};
    Align al;
    const int es = c.type == MOE_DTYPE_F32 ? 4 : 2;
    auto in = [&](const Matrix &m) {
        al.add(m.p, m.ld, c.d, es, c.T);
        return m.p;
    };
    auto out = [&](const Matrix &m) { return const_cast<void *>(in(m)); };
    a.x = in(c.x);
    a.ldx = c.x.ld;
    a.b = in(c.b);
    a.ldb = c.b.ld;
    a.full = c.gate.p != nullptr && c.gate_rows;
    a.gate = a.full ? in(c.gate) : c.gate.p;
    a.ldg = c.gate.ld;
    a.dy = in(c.dy);
    a.lddy = c.dy.ld;
    a.du = in(c.du);
    a.lddu = c.du.ld;
    a.dx = out(c.dx);
    a.lddx = c.dx.ld;
    a.db = out(c.db);
    a.lddb = c.db.ld;
    a.dgate = a.full ? out(c.dgate) : const_cast<void *>(c.dgate.p);
    a.lddg = c.dgate.ld;
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
    a.withheld = withheld;
    a.part = c.dpost != nullptr || c.dpre != nullptr ? c.part : nullptr;
    switch (c.type) {
        case MOE_DTYPE_BF16: return backward_type<__nv_bfloat16>(a, al, c.type, c.dpost, c.dpre, s);
        case MOE_DTYPE_F16: return backward_type<__half>(a, al, c.type, c.dpost, c.dpre, s);
        default: return backward_type<float>(a, al, c.type, c.dpost, c.dpre, s);
    }
}

}  // namespace moe
