// The norms around a block (block_norm.cuh), gradients, for one element type: with e = pre du,
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
//
// Measured, with the second kernel: 8192 x 7168 bf16 with a full gate 180 us (5.2 TB/s), 4096 x
// 4096 bf16 with a row's gate 45 us, 8192 x 4096 fp32 without one 138 us (5.8 TB/s); rows of 7167
// bf16, 300 us; 8192 x 14336 bf16 with a row's gate (pairs) 387 us (3.6 TB/s). The norm
// alone, 8192 x 7168 bf16: 77 us (4.6 TB/s), with the residual's gradient 86 (5.4); 4096 x 4096 27 and 30.
// One row group of 14 warps is all that the registers (the column sums and five values an element between the sums)
// let an SM hold of 7168 columns, and it waits twice a row for a sum.
#pragma once

#include <algorithm>
#include <type_traits>

#include "block_norm.cuh"

namespace moe {
namespace bn {
namespace {

constexpr int kBwdThreads = 512, kBwdFewThreads = 448;  // most of a block with a ring
constexpr size_t kPairCtl = (sizeof(PairCtl) + 127) / 128 * 128;
// Columns of the first CTA of a pair: half of the row's vectors, rounded up (so that the second
// half starts at the same place of 16 bytes as the row).
template <int V>
__host__ __device__ constexpr int half_columns(int d) { return ((d + V - 1) / V + 1) / 2 * V; }
__device__ __forceinline__ bool sum_lost(const GroupSum &) { return false; }
__device__ __forceinline__ bool sum_lost(const PairSum &s) { return s.dead; }

// Row `row` of the partial sums from a block's groups' [groups][2][n], in order: columns at .. at +
// cols - 1, which lie `lead` elements on.
__device__ __forceinline__ void add_groups(const Args &a, const float *sums, int n, int lead, int cols, int at,
                                           int row, int groups, bool lost) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
        const int m = c >= cols, i = c - m * cols;
        const float *from = sums + m * n + lead + i;
        float s = lost ? NAN : from[0];
        for (int k = 1; k < groups; ++k) s += from[(size_t)2 * k * n];
        a.part[((size_t)row * 2 + m) * a.d + at + i] = s;
    }
}

// Rows that no ring holds, straight from global memory: each pass forms again what it needs,
// from L1 or L2. All results are written by the last pass, after the thread's last read, so
// that they may replace inputs.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) backward_rows_kernel(const Args a) {
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
        // of a vector: yh, bh, g and 1 - g, du and dy
        float yh[V], bh[V], g[V], h[V], du[V], dy[V];
        auto form = [&](int v) {
            float x[V], z[V];
            load_row<T, V>(a.x, a.ldx, row, v, x);
            if (a.b != nullptr) load_row<T, V>(a.b, a.ldb, row, v, bh);
            if (a.full) load_row<T, V>(a.gate, a.ldg, row, v, z);
            if (a.pre_norm) load_row<T, V>(a.du, a.lddu, row, v, du);
            if (a.dy != nullptr) load_row<T, V>(a.dy, a.lddy, row, v, dy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[j] = g_row;
                h[j] = h_row;
                if (a.full) sigmoid(z[j], g[j], h[j]);
                float y = x[j];
                if (a.b != nullptr) {
                    bh[j] *= r_post;
                    y = fmaf(a.scale, y, g[j] * (bh[j] * load_w<T>(a.post, a.w32, v * V + j, 1.f)));
                } else {
                    bh[j] = 0.f;
                }
                yh[j] = y * r_pre;
                if (!a.pre_norm) du[j] = 0.f;
                if (a.dy == nullptr) dy[j] = 0.f;
            }
        };
        auto weight = [&](const void *w, int v, int j) { return load_w<T>(w, a.w32, v * V + j, 1.f); };
        float s = 0.f;
        if (a.pre_norm) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tpr + t;
                if (v >= nvec) continue;
                form(v);
#pragma unroll
                for (int j = 0; j < V; ++j) s = fmaf(du[j] * weight(a.pre, v, j), yh[j], s);
            }
        }
        const float c1 = a.pre_norm ? sum(s) * inv_d : 0.f;
        // dY of element j of vector v
        auto grad_y = [&](int v, int j) {
            return fmaf(r_pre, fmaf(-c1, yh[j], du[j] * weight(a.pre, v, j)), dy[j]);
        };
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t;
            if (v >= nvec) continue;
            form(v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gd = g[j] * grad_y(v, j) * bh[j];
                dpost[i][j] += gd;
                dpre[i][j] = fmaf(du[j], yh[j], dpre[i][j]);
                s = fmaf(gd, weight(a.post, v, j), s);
            }
        }
        if (a.b != nullptr) s = sum(s);
        const float c2 = a.post_norm ? s * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tpr + t;
            if (v >= nvec) continue;
            form(v);
            float dx[V], db[V], dz[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gy = grad_y(v, j), f = g[j] * gy * weight(a.post, v, j);
                dx[j] = a.b != nullptr ? a.scale * gy : gy;
                dz[j] = f * bh[j] * h[j];
                db[j] = r_post * fmaf(-c2, bh[j], f);
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
    add_groups(a, sums, a.d, 0, a.d, 0, blockIdx.x, groups, false);
}

template <typename T, int V, int NV>
cudaError_t backward_rows(Args a, int *P, cudaStream_t s) {
    RowShape r = row_shape(a, V * NV);
    r.grid = std::min(r.grid, kLnPartials);
    *P = r.grid;
    const size_t smem = a.part != nullptr ? (size_t)r.groups * 2 * a.d * sizeof(float) : 0;
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(backward_rows_kernel<T, V, NV>), (int)(2 * kBlockNormMaxWidth * sizeof(float)));
    if (e != cudaSuccess) return e;
    return launch_k(backward_rows_kernel<T, V, NV>, dim3(r.grid), dim3(r.groups * a.wpr * 32), smem, s, a);
}

// Rows through a ring, as the forward's. A stage holds x, b (MODE 1, 2) and the gate (MODE 2),
// then du and dy, where the call has them. MT: most threads. CTAS 2: a row is
// halved over a pair of CTAs, each with half of its threads and memory.
template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW, int MT, int CTAS>
__global__ void __launch_bounds__(MT, 1) backward_ring_kernel(const Args a) {
    extern __shared__ __align__(128) uint8_t ring_sh[];
    RingCtl *ctl = reinterpret_cast<RingCtl *>(ring_sh);
    using Wt = Weights<T, V, SHIFT, RAW>;
    constexpr int P2 = V / 2;
    const int tpr = a.wpr * 32, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int groups = blockDim.x / tpr, S = a.stages;
    const uint32_t rank = CTAS == 2 ? ptx::cluster_ctarank() : 0;
    const int unit = blockIdx.x / CTAS;
    const bool has_du = a.pre_norm, has_dy = a.dy != nullptr;
    const int K = MODE + 1 + has_du + has_dy;
    // the columns of this CTA's part: the first or the second half of the vectors, or all
    const int most = CTAS == 2 ? half_columns<V>(a.d) : a.d, first = rank * most, own = min(most, a.d - first);
    const uint32_t row_bytes = ring_row_bytes<T, SHIFT>(most);
    const uint32_t stage_bytes = K * row_bytes, w_bytes = Wt::bytes(most);
    const int64_t stride = (int64_t)(gridDim.x / CTAS) * groups;
    int64_t row = (int64_t)unit * groups + group;
    if (SHIFT) row = unit % kPhases + (int64_t)kPhases * (unit / kPhases * groups + group);
    // (the rows of a block start at the same place: its first row's, there or not)
    const Part<T, V, SHIFT> part(tpr, t, own, static_cast<T *>(a.dx) + unit % kPhases * a.lddx);
    PairCtl *pairs = reinterpret_cast<PairCtl *>(ring_sh + kRingCtl);
    uint8_t *post = ring_sh + kRingCtl + (CTAS == 2 ? kPairCtl : 0), *pre = post + (MODE > 0 ? w_bytes : 0);
    uint8_t *rings = pre + w_bytes;
    uint8_t *ring = rings + (size_t)group * a.group_bytes;
    const uint32_t bar0 = ptx::smem_addr(&ctl->full[group][0]);
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(bar0 + 8 * s, K + 1);
        if (CTAS == 2)
            for (int k = 0; k < 2; ++k) ptx::mbar_init(ptx::smem_addr(&pairs->bar[group][k]), 2 * a.wpr);
        ptx::fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    // row r of the stage's tensor k into stage s, or (k = K) its scalars: a thread each
    auto fetch = [&](int64_t r, int s, int k) {
        if (r == a.withheld) return;
        if (k == K) {
            fetch_scalars(ctl->scalars[group][s], has_du ? a.r_pre : nullptr,
                          MODE > 0 && a.post_norm ? a.r_post : nullptr, MODE == 1 ? static_cast<const float *>(a.gate) : nullptr, r, bar0 + 8 * s);
            return;
        }
        const void *p = a.x;
        int64_t ld = a.ldx;
        if (MODE > 0 && k == 1) p = a.b, ld = a.ldb;
        if (MODE > 1 && k == 2) p = a.gate, ld = a.ldg;
        if (k > MODE) {
            const bool u = has_du && k == MODE + 1;
            p = u ? a.du : a.dy;
            ld = u ? a.lddu : a.lddy;
        }
        fetch_row<T, SHIFT>(ring + (size_t)s * stage_bytes + (size_t)k * row_bytes, static_cast<const T *>(p) + first,
                            ld, r, a.T, own, bar0 + 8 * s);
    };
    __syncwarp();
    if (t < S * (K + 1) && row + t / (K + 1) * stride < a.T)
        fetch(row + t / (K + 1) * stride, t / (K + 1), t % (K + 1));
    if (MODE > 0) Wt::fill(post, a.post, a.w32, part, first);
    Wt::fill(pre, a.pre, a.w32, part, first);
    __syncthreads();
    if (CTAS == 2) ptx::cluster_sync();  // both CTAs' barriers are there

    f32x2 dpost[NV][P2], dpre[NV][P2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P2; ++j) dpost[i][j] = dpre[i][j] = 0;
    auto off = [&](const void *p, int64_t ld) { return part.off(static_cast<const T *>(p) + unit % kPhases * ld); };
    const int ox = off(a.x, a.ldx), ob = MODE > 0 ? off(a.b, a.ldb) : 0, oz = MODE > 1 ? off(a.gate, a.ldg) : 0;
    const int ou = has_du ? off(a.du, a.lddu) : 0, oy = has_dy ? off(a.dy, a.lddy) : 0;
    const int odx = 0, odb = MODE > 0 ? off(a.db, a.lddb) : 0, odz = MODE > 1 ? off(a.dgate, a.lddg) : 0;
    const float inv_d = 1.f / (float)a.d;
    using Sum = typename std::conditional<CTAS == 2, PairSum, GroupSum>::type;
    Sum sum = [&] {
        if constexpr (CTAS == 2) return PairSum{pairs, group, (int)(threadIdx.x >> 5) - group * a.wpr, a.wpr, rank};
        else return GroupSum{ctl->slots, group * a.wpr, a.wpr, 1 + group};
    }();
    int s = 0;
    uint32_t ph = 0;
    bool alive = true;
    for (; row < a.T; row += stride) {
        alive = alive && ring_wait(bar0, S, s, ph, t <= K);
        const float *scalars = ctl->scalars[group][s];
        float g_row = 1.f, h_row = 0.f;
        if (MODE == 1 && a.gate != nullptr) sigmoid(scalars[2], g_row, h_row);
        const float r_post = MODE > 0 && a.post_norm ? scalars[1] : 1.f, r_pre = has_du ? scalars[0] : 0.f;
        const uint8_t *stage = ring + (size_t)s * stage_bytes;
        auto image = [&](const void *p, int64_t ld) {
            return image_at<T, SHIFT>(static_cast<const T *>(p) + first, ld, row);
        };
        const uint8_t *px = stage + image(a.x, a.ldx);
        const uint8_t *pb = stage + row_bytes + (MODE > 0 ? image(a.b, a.ldb) : 0);
        const uint8_t *pz = stage + 2 * row_bytes + (MODE > 1 ? image(a.gate, a.ldg) : 0);
        const uint8_t *pu = stage + (MODE + 1) * row_bytes + image(a.du, a.lddu);
        const uint8_t *py = stage + (MODE + 1 + has_du) * row_bytes + image(a.dy, a.lddy);
        // (a row that did not come: NaN)
        const f32x2 scale = both(alive ? a.scale : NAN), rp = both(alive ? r_post : NAN), rq = both(r_pre);
        // yh, then f; g and 1 - g, then bh
        f32x2 yh[NV][P2], g[NV][P2], h[MODE == 2 ? NV : 1][P2], q = alive ? 0 : both(NAN);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!part.has(i)) continue;
            f32x2 w[P2], du[P2];
            part.load(px, ox, i, yh[i]);
            if (MODE > 0) {
                f32x2 b[P2];
                part.load(pb, ob, i, b);
                Wt::load(part, post, i, w);
                if (MODE == 2) {
                    f32x2 z[P2];
                    part.load(pz, oz, i, z);
#pragma unroll
                    for (int j = 0; j < P2; ++j) sigmoid2<T, true>(z[j], g[i][j], h[i][j]);
                }
#pragma unroll
                for (int j = 0; j < P2; ++j)
                    yh[i][j] = fma2(scale, yh[i][j], mul2(mul2(mul2(b[j], rp), w[j]), MODE == 2 ? g[i][j] : both(g_row)));
            }
            if (has_du) {
                part.load(pu, ou, i, du);
                Wt::load(part, pre, i, w);
#pragma unroll
                for (int j = 0; j < P2; ++j) {
                    yh[i][j] = mul2(yh[i][j], rq);
                    dpre[i][j] = fma2(du[j], yh[i][j], dpre[i][j]);
                    q = fma2(mul2(du[j], w[j]), yh[i][j], q);
                }
            }
        }
        const f32x2 c1 = both(has_du ? -sum(pair_sum(q)) * inv_d : 0.f);
        q = alive ? 0 : both(NAN);
        T *xrow = static_cast<T *>(a.dx) + row * a.lddx + first;
        T *brow = static_cast<T *>(a.db) + row * a.lddb + first;
        T *zrow = static_cast<T *>(a.dgate) + row * a.lddg + first;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!part.has(i)) continue;
            f32x2 w[P2], d[P2];
            // dY
#pragma unroll
            for (int j = 0; j < P2; ++j) d[j] = 0;
            if (has_dy) part.load(py, oy, i, d);
            if (has_du) {
                f32x2 du[P2];
                part.load(pu, ou, i, du);
                Wt::load(part, pre, i, w);
#pragma unroll
                for (int j = 0; j < P2; ++j) d[j] = fma2(rq, fma2(yh[i][j], c1, mul2(du[j], w[j])), d[j]);
            }
            if (MODE == 0) {
                part.store(xrow, odx, i, d);
                continue;
            }
            f32x2 b[P2], o[P2];
            part.load(pb, ob, i, b);
            Wt::load(part, post, i, w);
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                o[j] = mul2(scale, d[j]);
                d[j] = mul2(d[j], MODE == 2 ? g[i][j] : both(g_row));
                b[j] = mul2(b[j], rp);
                dpost[i][j] = fma2(d[j], b[j], dpost[i][j]);
                d[j] = mul2(d[j], w[j]);  // f
            }
            part.store(xrow, odx, i, o);
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                const f32x2 fb = mul2(d[j], b[j]);
                q = add2(q, fb);
                if (MODE == 2) o[j] = mul2(fb, h[i][j]);
                yh[i][j] = d[j];
                g[i][j] = b[j];
            }
            if (MODE == 2) part.store(zrow, odz, i, o);
        }
        float ss = 0.f;
        if (MODE > 0) ss = sum(pair_sum(q));
        else if (a.wpr > 1) group_sync(1 + group, tpr);
        if (a.wpr == 1) __syncwarp();
        // every thread of the group is done with the stage
        if (t <= K && alive && row + S * stride < a.T) fetch(row + S * stride, s, t);
        if (MODE > 0) {
            if (MODE == 1 && t == 0 && rank == 0 && a.gate != nullptr) static_cast<float *>(a.dgate)[row] = h_row * ss;
            const f32x2 c2 = both(a.post_norm ? -ss * inv_d : 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!part.has(i)) continue;
                f32x2 o[P2];
#pragma unroll
                for (int j = 0; j < P2; ++j) o[j] = mul2(rp, fma2(g[i][j], c2, yh[i][j]));
                part.store(brow, odb, i, o);
            }
        }
        if (++s == S) {
            s = 0;
            ph ^= 1;
        }
    }
    if (CTAS == 2) {  // nothing of this CTA is on its way to the other, or back
        __syncwarp();
        ptx::cluster_sync();
    }
    if (a.part == nullptr) return;
    if constexpr (!SHIFT && CTAS == 1) {
        bool ok[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) ok[i] = part.has(i);
        store_partials<V, NV>(a.part, a.d, groups, group, tpr, t, ok, dpost, dpre, rings, a.group_bytes, !alive);
    } else {
        // every thread is done with the last rows
        const bool lost = __syncthreads_or(!alive || sum_lost(sum));
        float *sums = reinterpret_cast<float *>(rings);  // [groups][2][nvec V], `lead` columns on
        const int n = part.nvec * V;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!part.has(i)) continue;
            f32x2 *at = reinterpret_cast<f32x2 *>(sums + (size_t)2 * group * n + (i * tpr + t) * V);
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                at[j] = dpost[i][j];
                at[n / 2 + j] = dpre[i][j];
            }
        }
        add_groups(a, sums, n, part.lead, part.d, first, unit, groups, lost);
    }
}

template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW, int CTAS>
bool backward_shape(Args &a, int threads, int *groups, size_t *smem) {
    const int cols = CTAS == 2 ? half_columns<V>(a.d) : a.d;
    const size_t stage = (MODE + 1 + a.pre_norm + (a.dy != nullptr)) * ring_row_bytes<T, SHIFT>(cols);
    const size_t fixed =
        kRingCtl + (CTAS == 2 ? kPairCtl : 0) + (MODE > 0 ? 2 : 1) * Weights<T, V, SHIFT, RAW>::bytes(cols);
    // (a group's ring holds its fp32 sums in the end, [2][d] and up to two vectors more, in whole
    // lines: 128 bytes more than two stages of two 16-bit tensors, those of the norm alone. A rule that
    // had the stages hold them sent its aligned rows past the ring: 8192 x 7168 bf16 615 / 77 us)
    const size_t sums = (2 * ((size_t)cols + 2 * V) * sizeof(float) + 127) / 128 * 128;
    if (!shape_of(a, ring_cols<V, SHIFT>(cols), V * NV, threads, sm_count() / CTAS, fixed, stage, sums, groups))
        return false;
    *smem = fixed + (size_t)*groups * a.group_bytes;
    return true;
}
// The block of at most 448 threads is compiled for as many registers as that of 512 (128), but
// runs up to 6 % faster where both have the same groups, or nearly (8192 x 7168 bf16 with a row's
// gate 137 / 145 us, with a full one 182 / 179, 4096 x 1024 21.6 / 22.7; 4096 x 4096 with a row's,
// one group against two, 58 / 45).
template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW>
bool backward_best(Args &a, int *threads, int *groups, size_t *smem) {
    Args few = a;
    int g = 0;
    size_t m = 0;
    *threads = kBwdThreads;
    const bool fits = backward_shape<T, V, NV, MODE, SHIFT, RAW, 1>(a, kBwdThreads, groups, smem);
    if (fits && backward_shape<T, V, NV, MODE, SHIFT, RAW, 1>(few, kBwdFewThreads, &g, &m) && 5 * g >= 4 * *groups) {
        a = few;
        *threads = kBwdFewThreads;
        *groups = g;
        *smem = m;
    }
    return fits;
}
template <typename T, int V, int NV, int MODE, int SHIFT, bool RAW>
cudaError_t backward_launch(const Args &a, int threads, int groups, size_t smem, int *P, cudaStream_t s) {
    const auto kernel = threads == kBwdFewThreads
                            ? backward_ring_kernel<T, V, NV, MODE, SHIFT, RAW, kBwdFewThreads, 1>
                            : backward_ring_kernel<T, V, NV, MODE, SHIFT, RAW, kBwdThreads, 1>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)kRingSmem);
    if (e != cudaSuccess) return e;
    *P = ring_grid<SHIFT>(a.T, groups, std::min(sm_count(), kLnPartials));
    return launch_k(kernel, dim3(*P), dim3(groups * a.wpr * 32), smem, s, a);
}
// Weights as in the forward; the fullest form of rows that start anywhere spills less without planes
// (8192 x 7167 bf16 with a full gate 326 us with, 300 without, 4096 x 5001 135 / 129; with a
// row's gate 214 / 220).
template <typename T, int MODE, int SHIFT>
cudaError_t backward_ring(const Args &a, int *P, bool *fits, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T), NV = 16 / V;  // 16 elements a thread
    Args planes = a;
    int groups = 0, threads = 0;
    size_t smem = 0;
    *fits = backward_best<T, V, NV, MODE, SHIFT, false>(planes, &threads, &groups, &smem);
    if constexpr (sizeof(T) == 2) {
        Args raw = a;
        int more = 0, t = 0;
        size_t less = 0;
        if (!a.w32 && backward_best<T, V, NV, MODE, SHIFT, true>(raw, &t, &more, &less) &&
            (!*fits || rows_ahead(raw, more) + (SHIFT && MODE == 2) > rows_ahead(planes, groups))) {
            *fits = true;
            return backward_launch<T, V, NV, MODE, SHIFT, true>(raw, t, more, less, P, s);
        }
    }
    if (*fits) return backward_launch<T, V, NV, MODE, SHIFT, false>(planes, threads, groups, smem, P, s);
    // Rows that no SM holds: halves, over pairs of CTAs (8192 x 14336 bf16 with a row's gate
    // 1580 / 387 us without and with, 4096 x 14335 1849 / 260; where an SM holds one row, two
    // halves of two rows in its place are slower: 8192 x 7168 bf16 with a full gate 180 / 235).
    Args pair = a;
    if (!backward_shape<T, V, NV, MODE, SHIFT, false, 2>(pair, kBwdThreads, &groups, &smem)) return cudaSuccess;
    *fits = true;
    const auto kernel = backward_ring_kernel<T, V, NV, MODE, SHIFT, false, kBwdThreads, 2>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)kRingSmem);
    if (e != cudaSuccess) return e;
    *P = ring_grid<SHIFT>(a.T, groups, std::min(sm_count() / 2, kLnPartials));
    return launch_pairs(kernel, dim3(2 * *P), dim3(groups * pair.wpr * 32), smem, s, pair);
}
template <typename T, int SHIFT>
cudaError_t backward_rings(const Args &a, int *P, bool *fits, cudaStream_t s) {
    return a.b == nullptr ? backward_ring<T, 0, SHIFT>(a, P, fits, s)
           : !a.full      ? backward_ring<T, 1, SHIFT>(a, P, fits, s)
                          : backward_ring<T, 2, SHIFT>(a, P, fits, s);
}

}  // namespace

template <typename T>
cudaError_t backward_type(const Args &a, int shift, int *P, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    bool fits = false;
    const cudaError_t e = shift == 0   ? backward_rings<T, 0>(a, P, &fits, s)
                          : shift == 1 ? backward_rings<T, 1>(a, P, &fits, s)
                                       : backward_rings<T, 2>(a, P, &fits, s);
    if (e != cudaSuccess || fits) return e;
    return shift == 0 ? backward_rows<T, W, 16 / W>(a, P, s) : backward_rows<T, 1, 16>(a, P, s);
}

}  // namespace bn
}  // namespace moe
