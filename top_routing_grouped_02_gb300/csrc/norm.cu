// Layer norm, forward and backward.
//
//   y = gamma (x - m) r + beta,  m = mean of the row, r = 1 / sqrt(var + eps)
//   g = gamma dy,  xh = (x - m) r
//   dx = r (g - mean(g) - xh mean(g xh))  (+ dres)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both are bound by HBM: the forward reads x and writes y once, the backward
// reads x, dy (and dres) and writes dx once. A group of warps takes a row at a time
// from a ring of rows in shared memory, which is filled asynchronously ahead of it.
// Measured, calls back to back, 8192 x 7168 bf16: forward 40 us (5.9 TB/s), backward with
// dres and the sum of the weights' partials 87 us (5.4 TB/s); rows of 7167: 65 and 141 us
// (109 without dres), bound by the shifts' instructions; 4096 x 4096: 15 and 28 us, of
// which some 6 and 10 are the starts and ends of the kernels. The partials' sum takes 4.
//
// Row statistics: each warp takes the mean and the squared deviations from its own mean
// of its elements, and the warps' pairs are joined by
//   m = sum n_w m_w / d,  M2 = sum (M2_w + n_w (m_w - m)^2),
// one exchange through shared memory a row, with no subtraction of large equal
// numbers: a row whose offset is far larger than its spread keeps its variance (to within
// 2^-24 of their ratio: the warps' means are rounded; y is off by as much through m). The
// backward takes x - m before it scales, for the same reason.
//
// Weight gradients: each thread owns its columns and sums them over the rows of
// its group in fp32 registers; the groups of a block are added in a fixed order
// through shared memory, each block writes one partial row per array, and a
// second kernel adds the blocks' partials in a fixed order. No atomics: the
// result does not depend on timing.
//
// Rows too wide for a ring take kernels that read the row again from L2 for each
// pass.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Threads of a ring block: 72 registers a thread forward, 128 backward, where the
// column sums take 64.
constexpr int kFwdThreads = 896, kBwdRingThreads = 512;

struct LnArgs {
    const void *x, *gamma, *beta;
    void *y;
    float *mean, *rstd;
    int64_t ldx, ldy;
    int64_t T;
    int d;
    int w32;  // gamma, beta (and their gradients) are fp32, else x's type
    float eps;
    int wpr;  // warps per row
    int stages;  // ring stages per row group
    int64_t withheld;  // self-test: this row's copies are never issued (-1: none)
    // backward
    const void *dy, *dres;
    void *dx;
    int64_t lddy, lddres, lddx;
    float *part;       // [blocks][2][d] partial sums (dgamma, dbeta), or NULL
};

template <typename T>
__device__ __forceinline__ float load_w(const void *w, int w32, int c, float none) {
    if (w == nullptr) return none;
    return w32 ? static_cast<const float *>(w)[c] : load_f32(static_cast<const T *>(w) + c);
}

// Elements of a row that warp w of `tpr` threads holds, NV vectors of V each thread.
template <int V, int NV>
__device__ __forceinline__ int warp_count(int w, int nvec, int tpr) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) n += min(max(nvec - (i * tpr + w * 32), 0), 32);
    return n * V;
}

// ---- a ring of rows in shared memory ---------------------------------------------
//
// Each row group keeps a ring of its next rows in shared memory, filled by bulk
// copies (cp.async.bulk, issued by the group's first threads, completion on an mbarrier), so
// that the loads in flight do not depend on how far the group's arithmetic is and
// take no registers. A stage is refilled after a barrier that every thread of the
// group passes after its last read of the stage.
//
// With that the kernels are limited by instruction issue nearly as much as by HBM,
// so a row is spread over few threads (V * NV = 32 elements of 16 bits each: the
// shuffles, barrier and bookkeeping of a row are paid per warp), the arithmetic is
// on packed pairs, and gamma and beta wait in shared memory in fp32, as planes of
// four elements of every vector, which a warp reads without bank conflicts.
//
// SHIFT: rows that do not start on 16-byte boundaries (an odd length, a sliced
// buffer). The bulk copies take the 16-byte blocks that hold a row, so its image starts
// up to 15 bytes into the stage, and a thread shifts its vectors out of two
// neighbouring ones; results go to an image of the output row in shared memory, which
// leaves by a bulk copy of its whole blocks and by element at its ends. Nothing is
// read before the first or after the last element of a tensor: there the row's ends
// come by element too.

constexpr int kRingStages = 4;  // most
constexpr int kMaxGroups = 28;
struct RingCtl {
    uint64_t full[kMaxGroups][kRingStages];
    float2 stat[2][32];
    uint4 zero;  // what a thread past the row's end reads
};
constexpr int kRingCtl = (sizeof(RingCtl) + 127) / 128 * 128;
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// Waits for stage s. A copy that has not arrived after about a second never will (it was
// issued by this block: the device has stopped). Then false, and the caller's group gives
// up: it issues no further copies, its rows' results and the block's sums become NaN. Copies
// in flight land before the block leaves, as far as another limit allows (drain: the
// threads that issue copies wait for them).
__device__ __noinline__ bool ring_wait_long(uint32_t bar0, int stages, int s, uint32_t parity, bool drain) {
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

// A block's partial sums dgamma, dbeta: each group puts its own into its ring (as planes,
// [2][d rounded up to V]), and the block adds the groups' in order, four columns a
// thread. (One group after the other through one copy took 3.5 us for 4 groups of d =
// 4096.)
template <int V, int NV>
__device__ __forceinline__ void store_partials(const LnArgs &a, int groups, int group, int tpr,
                                               int t, const bool (&ok)[NV],
                                               const f32x2 (&dg)[NV][V / 2],
                                               const f32x2 (&db)[NV][V / 2], uint8_t *rings,
                                               size_t ring_bytes, bool gave_up) {
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    const int nvec = (a.d + V - 1) / V;
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
        if (4 * e >= a.d) continue;  // the last vector may reach past the row
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
        float *out = part + (int64_t)m * a.d + 4 * e;
        if ((a.d & 3) == 0) {
            *reinterpret_cast<float4 *>(out) = x;
        } else {
            const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * e + j < a.d) out[j] = f[j];
        }
    }
}

// ---- SHIFT helpers

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
// v's first n elements (of 16 bytes), zeros after them.
template <typename T>
__device__ __forceinline__ uint4 first_elems(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int left = (int)(n * sizeof(T)) - 4 * j;  // bytes of this word
        if (left <= 0) w[j] = 0;
        else if (left == 2) w[j] &= 0xffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Writes n elements of a vector into the image of an output row.
template <typename T>
__device__ __forceinline__ void put_image(uint8_t *img, int v, uint32_t shift, uint4 q, int n) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint8_t *p = img + shift + v * 16;
    if (n * (int)sizeof(T) == 16) {
        if (sizeof(T) == 4 || (shift & 2) == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t *>(p)[j] = w[j];
        } else {
            *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
#pragma unroll
            for (int j = 0; j < 3; ++j)
                *reinterpret_cast<uint32_t *>(p + 2 + 4 * j) = __funnelshift_r(w[j], w[j + 1], 16);
            *reinterpret_cast<uint16_t *>(p + 14) = (uint16_t)(w[3] >> 16);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 16 / (int)sizeof(T); ++e)
        if (e < n) {
            if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(p)[e] = w[e];
            else reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
}
// An output row from its image: whole blocks by one bulk copy (thread 0), the
// elements at its ends by the group's other threads.
template <typename T>
__device__ __forceinline__ void send_image(const uint8_t *img, T *row, int d, int t, int tpr) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row), end = reinterpret_cast<uintptr_t>(row + d);
    const uintptr_t origin = at & ~(uintptr_t)15;
    const uintptr_t lo = (at + 15) & ~(uintptr_t)15, hi = end & ~(uintptr_t)15;
    const bool whole = hi > lo;
    if (t == 0) {
        if (whole)
            ptx::bulk_store(reinterpret_cast<void *>(lo), ptx::smem_addr(img + (lo - origin)),
                            (uint32_t)(hi - lo));
        ptx::bulk_commit_group();
    }
    const T *from = reinterpret_cast<const T *>(img + (at - origin));
    const int head = whole ? (int)((lo - at) / sizeof(T)) : d;
    const int tail = whole ? (int)((end - hi) / sizeof(T)) : 0;
    for (int i = t; i < head + tail; i += tpr) {
        const int e = i < head ? i : d - tail + (i - head);
        row[e] = from[e];
    }
}

template <typename T, int V, int NV, bool SHIFT>
__global__ void __launch_bounds__(kFwdThreads, 1) ln_forward_ring_kernel(const LnArgs a) {
    extern __shared__ __align__(128) uint8_t ring_sh[];
    RingCtl *ctl = reinterpret_cast<RingCtl *>(ring_sh);
    constexpr int P2 = V / 2;
    const int tpr = a.wpr * 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int w0 = group * a.wpr, wg = warp - w0;
    const int groups = blockDim.x / tpr, S = a.stages;
    const int nvec = (a.d + V - 1) / V;
    const uint32_t row_bytes = SHIFT ? image_bytes(a.d, sizeof(T)) : (uint32_t)a.d * sizeof(T);
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    float *gamma = reinterpret_cast<float *>(ring_sh + kRingCtl), *beta = gamma + nvec * V;
    // a group's ring and (SHIFT) its output image
    uint8_t *ring = ring_sh + kRingCtl + (size_t)2 * nvec * V * sizeof(float) +
                    (size_t)group * (S + SHIFT) * row_bytes;
    uint8_t *image = ring + (size_t)S * row_bytes;
    const uint32_t bar0 = ptx::smem_addr(&ctl->full[group][0]);
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(bar0 + 8 * s, 1);
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) ctl->zero = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](int64_t r, int s) {
        if (r == a.withheld) return;
        if constexpr (SHIFT) {
            const uint32_t bytes = fetch_image(ring + (size_t)s * row_bytes, static_cast<const T *>(a.x),
                                               a.ldx, r, a.T, a.d, bar0 + 8 * s);
            ptx::mbar_arrive_expect_tx(bar0 + 8 * s, bytes);
            return;
        }
        ptx::mbar_arrive_expect_tx(bar0 + 8 * s, row_bytes);
        ptx::bulk_load(ptx::smem_addr(ring + (size_t)s * row_bytes),
                       static_cast<const T *>(a.x) + r * a.ldx, row_bytes, bar0 + 8 * s);
    };
    // (a stage a thread: their addresses and issue take 0.3 to 0.6 us each)
    __syncwarp();
    if (t < S && row + t * stride < a.T) fetch(row + t * stride, t);
    fill_planes<T, V>(gamma, a.gamma, a.w32, a.d, 1.f);
    fill_planes<T, V>(beta, a.beta, a.w32, a.d, 0.f);
    __syncthreads();

    bool ok[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) ok[i] = i * tpr + t < nvec;
    const float inv_d = 1.f / (float)a.d;
    // elements of a warp: its vectors, less what the last one lacks
    const int lacks = nvec * V - a.d, last = (nvec - 1) % tpr / 32;
    const int n_own = warp_count<V, NV>(wg, nvec, tpr) - (wg == last ? lacks : 0);
    const float inv_own = n_own > 0 ? 1.f / (float)n_own : 0.f;
    const float n_lane =
        lane < a.wpr ? (float)(warp_count<V, NV>(lane, nvec, tpr) - (lane == last ? lacks : 0)) : 0.f;

    int s = 0;
    uint32_t ph = 0;
    bool alive = true;
    for (int buf = 0; row < a.T; row += stride, buf ^= 1) {
        alive = alive && ring_wait(bar0, S, s, ph, t == 0);
        const uint8_t *stage = ring + (size_t)s * row_bytes;
        const uint4 *src = reinterpret_cast<const uint4 *>(stage) + t;
        const uint32_t sx = (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const T *>(a.x) + row * a.ldx) & 15;
        // f: the elements, then their distances from the warp's own mean (a thread past
        // the row's end holds zeros throughout)
        f32x2 f[NV][P2], acc = alive ? 0 : both(NAN);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (SHIFT) {
                const int v = i * tpr + t;
                uint4 q = ok[i] ? image_vec<T>(stage, v, sx) : make_uint4(0, 0, 0, 0);
                if ((v + 1) * V > a.d) q = first_elems<T>(q, a.d - v * V);
                to_pairs<T, V>(q, f[i]);
            } else {
                to_pairs<T, V>(ok[i] ? src[i * tpr] : ctl->zero, f[i]);
            }
#pragma unroll
            for (int j = 0; j < P2; ++j) acc = add2(acc, f[i][j]);
        }
        const float own = warp_sum(pair_sum(acc)) * inv_own;
        acc = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const f32x2 shift = both(ok[i] ? -own : 0.f);
            if (SHIFT && ok[i] && (i * tpr + t + 1) * V > a.d) {
                // the last vector: what it lacks stays zero
                const int n = a.d - (i * tpr + t) * V;
#pragma unroll
                for (int j = 0; j < P2; ++j) {
                    f[i][j] = add2(f[i][j], pair(2 * j < n ? -own : 0.f, 2 * j + 1 < n ? -own : 0.f));
                    acc = fma2(f[i][j], f[i][j], acc);
                }
                continue;
            }
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                f[i][j] = add2(f[i][j], shift);
                acc = fma2(f[i][j], f[i][j], acc);
            }
        }
        float mean = own, dev = warp_sum(pair_sum(acc));
        if (SHIFT && t == 0) ptx::bulk_wait_group_read<0>();  // the image may be written again
        if (a.wpr > 1) {
            if (lane == 0) ctl->stat[buf][warp] = make_float2(own, dev);
            group_sync(1 + group, tpr);
        } else {
            __syncwarp();
        }
        // every thread of the group has read the stage
        if (t == 0 && alive && row + S * stride < a.T) fetch(row + S * stride, s);
        if (++s == S) {
            s = 0;
            ph ^= 1;
        }
        if (a.wpr > 1) {
            const float2 o = lane < a.wpr ? ctl->stat[buf][w0 + lane] : make_float2(0.f, 0.f);
            mean = warp_sum(n_lane * o.x) * inv_d;
            const float c = o.x - mean;
            dev = warp_sum(n_lane > 0.f ? fmaf(n_lane * c, c, o.y) : 0.f);
        }
        const float rstd = __frsqrt_rn(fmaf(dev, inv_d, a.eps));
        const f32x2 r2 = both(rstd), off = both((own - mean) * rstd);
        T *yrow = static_cast<T *>(a.y) + row * a.ldy;
        uint4 *yp = reinterpret_cast<uint4 *>(yrow) + t;
        const uint32_t sy = (uint32_t)reinterpret_cast<uintptr_t>(yrow) & 15;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!ok[i]) continue;
            f32x2 g[P2], o[P2];
            plane_pairs<V>(gamma, nvec, i * tpr + t, g);
            plane_pairs<V>(beta, nvec, i * tpr + t, o);
#pragma unroll
            for (int j = 0; j < P2; ++j) o[j] = fma2(fma2(f[i][j], r2, off), g[j], o[j]);
            const uint4 q = from_pairs<T, V>(o);
            if constexpr (SHIFT) put_image<T>(image, i * tpr + t, sy, q, min(V, a.d - (i * tpr + t) * V));
            else yp[i * tpr] = q;
        }
        if constexpr (SHIFT) {
            ptx::fence_proxy_async_smem();
            if (a.wpr > 1) group_sync(1 + group, tpr);
            else __syncwarp();
            send_image(image, yrow, a.d, t, tpr);
        }
        if (t == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
    }
    if (SHIFT && t == 0) ptx::bulk_wait_group<0>();
}

template <typename T, int V, int NV, bool SHIFT>
__global__ void __launch_bounds__(kBwdRingThreads, 1) ln_backward_ring_kernel(const LnArgs a) {
    extern __shared__ __align__(128) uint8_t ring_sh[];
    RingCtl *ctl = reinterpret_cast<RingCtl *>(ring_sh);
    constexpr int P2 = V / 2;
    const int tpr = a.wpr * 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
    const int w0 = group * a.wpr;
    const int groups = blockDim.x / tpr, S = a.stages;
    const int nvec = (a.d + V - 1) / V;
    const uint32_t row_bytes = SHIFT ? image_bytes(a.d, sizeof(T)) : (uint32_t)a.d * sizeof(T);
    const bool has_res = a.dres != nullptr;
    const int tensors = has_res ? 3 : 2;
    const uint32_t stage_bytes = tensors * row_bytes;
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    // gamma, then the rings, where the sums of the groups go in the end
    float *gamma = reinterpret_cast<float *>(ring_sh + kRingCtl);
    uint8_t *rings = ring_sh + kRingCtl + (size_t)nvec * V * sizeof(float);
    uint8_t *ring = rings + (size_t)group * (S * stage_bytes + SHIFT * row_bytes);
    uint8_t *image = ring + (size_t)S * stage_bytes;
    const uint32_t bar0 = ptx::smem_addr(&ctl->full[group][0]);
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(bar0 + 8 * s, tensors);
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) ctl->zero = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    // row r of tensor k (x, dy, dres) into stage s: a thread each
    auto fetch = [&](int64_t r, int s, int k) {
        if (r == a.withheld) return;
        const uint32_t bar = bar0 + 8 * s;
        uint8_t *dst = ring + (size_t)s * stage_bytes + (size_t)k * row_bytes;
        const T *base = static_cast<const T *>(k == 0 ? a.x : k == 1 ? a.dy : a.dres);
        const int64_t ld = k == 0 ? a.ldx : k == 1 ? a.lddy : a.lddres;
        if constexpr (SHIFT) {
            const uint32_t bytes = fetch_image(dst, base, ld, r, a.T, a.d, bar);
            ptx::mbar_arrive_expect_tx(bar, bytes);
        } else {
            ptx::mbar_arrive_expect_tx(bar, row_bytes);
            ptx::bulk_load(ptx::smem_addr(dst), base + r * ld, row_bytes, bar);
        }
    };
    __syncwarp();
    if (t < S * tensors) {
        const int s = t / tensors;
        if (row + s * stride < a.T) fetch(row + s * stride, s, t - s * tensors);
    }
    fill_planes<T, V>(gamma, a.gamma, a.w32, a.d, 1.f);
    __syncthreads();

    bool ok[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) ok[i] = i * tpr + t < nvec;
    f32x2 dg[NV][P2], db[NV][P2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P2; ++j) dg[i][j] = db[i][j] = 0;
    const float inv_d = 1.f / (float)a.d;
    float m_next = 0.f, r_next = 0.f;
    if (row < a.T) {
        m_next = a.mean[row];
        r_next = a.rstd[row];
    }

    int s = 0, s_prev = -1;
    uint32_t ph = 0;
    bool alive = true;
    for (int buf = 0; row < a.T; row += stride, buf ^= 1) {
        const float mean = m_next, rstd = r_next;
        if (row + stride < a.T) {
            m_next = a.mean[row + stride];
            r_next = a.rstd[row + stride];
        }
        alive = alive && ring_wait(bar0, S, s, ph, t < tensors);
        const uint8_t *stage = ring + (size_t)s * stage_bytes;
        const uint4 *px = reinterpret_cast<const uint4 *>(stage) + t;
        const uint4 *py = px + nvec, *pr = py + nvec;
        // vector i of x, dy, dres
        auto shift_of = [&](const void *base, int64_t ld) {
            return (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const T *>(base) + row * ld) & 15;
        };
        const uint32_t sx = shift_of(a.x, a.ldx), sy = shift_of(a.dy, a.lddy), sr = shift_of(a.dres, a.lddres);
        auto vec_x = [&](int i) { return SHIFT ? image_vec<T>(stage, i * tpr + t, sx) : px[i * tpr]; };
        auto vec_y = [&](int i) { return SHIFT ? image_vec<T>(stage + row_bytes, i * tpr + t, sy) : py[i * tpr]; };
        auto vec_r = [&](int i) { return SHIFT ? image_vec<T>(stage + 2 * row_bytes, i * tpr + t, sr) : pr[i * tpr]; };
        // xh = (x - m) r, the difference first: of x r and m r, both far larger where the
        // row's offset is far above its spread, nothing but rounding would be left (one
        // operation a pair and pass: 8192 x 7168 bf16 86.1 -> 86.5 us, 7167 137 -> 141)
        const f32x2 r2 = both(rstd), shift = both(-mean);
        f32x2 p1 = 0, p2 = alive ? 0 : both(NAN);
        constexpr bool KEEP = sizeof(T) == 4;  // xh and dy stay in registers (16 bits: too many)
        f32x2 kx[KEEP ? NV : 1][P2], ky[KEEP ? NV : 1][P2];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!ok[i]) continue;
            f32x2 (&x)[P2] = kx[KEEP ? i : 0], (&y)[P2] = ky[KEEP ? i : 0], g[P2];
            uint4 qx = vec_x(i), qy = vec_y(i);
            if (SHIFT && (i * tpr + t + 1) * V > a.d) {  // what the last vector lacks adds nothing
                qx = first_elems<T>(qx, a.d - (i * tpr + t) * V);
                qy = first_elems<T>(qy, a.d - (i * tpr + t) * V);
            }
            to_pairs<T, V>(qx, x);
            to_pairs<T, V>(qy, y);
            plane_pairs<V>(gamma, nvec, i * tpr + t, g);
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                const f32x2 gy = mul2(y[j], g[j]);
                x[j] = mul2(add2(x[j], shift), r2);
                db[i][j] = add2(db[i][j], y[j]);
                dg[i][j] = fma2(y[j], x[j], dg[i][j]);
                p2 = add2(p2, gy);
                p1 = fma2(gy, x[j], p1);
            }
        }
        float s1 = warp_sum(pair_sum(p1)), s2 = warp_sum(pair_sum(p2));
        if (SHIFT && t == 0) ptx::bulk_wait_group_read<0>();  // the image may be written again
        if (a.wpr > 1) {
            if (lane == 0) ctl->stat[buf][warp] = make_float2(s1, s2);
            group_sync(1 + group, tpr);
        } else {
            __syncwarp();
        }
        // every thread of the group is done with the previous row's stage
        if (!SHIFT && t < tensors && alive && s_prev >= 0 && row + (S - 1) * stride < a.T)
            fetch(row + (S - 1) * stride, s_prev, t);
        if (a.wpr > 1) {
            const float2 o = lane < a.wpr ? ctl->stat[buf][w0 + lane] : make_float2(0.f, 0.f);
            s1 = warp_sum(o.x);
            s2 = warp_sum(o.y);
        }
        // dx = gy r - xh (c1 r) - c2 r
        const f32x2 k1 = both(-s1 * inv_d * rstd), k2 = both(-s2 * inv_d * rstd);
        T *drow = static_cast<T *>(a.dx) + row * a.lddx;
        uint4 *pd = reinterpret_cast<uint4 *>(drow) + t;
        const uint32_t sd = (uint32_t)reinterpret_cast<uintptr_t>(drow) & 15;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!ok[i]) continue;
            f32x2 (&x)[P2] = kx[KEEP ? i : 0], (&y)[P2] = ky[KEEP ? i : 0], g[P2];
            if (!KEEP) {
                to_pairs<T, V>(vec_x(i), x);
                to_pairs<T, V>(vec_y(i), y);
            }
            plane_pairs<V>(gamma, nvec, i * tpr + t, g);
#pragma unroll
            for (int j = 0; j < P2; ++j) {
                if (!KEEP) x[j] = mul2(add2(x[j], shift), r2);
                x[j] = fma2(x[j], k1, fma2(mul2(y[j], g[j]), r2, k2));
            }
            if (has_res) {
                to_pairs<T, V>(vec_r(i), y);
#pragma unroll
                for (int j = 0; j < P2; ++j) x[j] = add2(x[j], y[j]);
            }
            const uint4 q = from_pairs<T, V>(x);
            if constexpr (SHIFT) put_image<T>(image, i * tpr + t, sd, q, min(V, a.d - (i * tpr + t) * V));
            else pd[i * tpr] = q;
        }
        if constexpr (SHIFT) {
            ptx::fence_proxy_async_smem();
            if (a.wpr > 1) group_sync(1 + group, tpr);
            else __syncwarp();
            // every thread of the group is done with this row's stage
            if (t < tensors && alive && row + S * stride < a.T) fetch(row + S * stride, s, t);
            send_image(image, drow, a.d, t, tpr);
        }
        s_prev = s;
        if (++s == S) {
            s = 0;
            ph ^= 1;
        }
    }
    if (SHIFT && t == 0) ptx::bulk_wait_group<0>();
    if (a.part == nullptr) return;
    store_partials<V, NV>(a, groups, group, tpr, t, ok, dg, db, rings, S * stage_bytes + SHIFT * row_bytes,
                          !alive);
}

// dgamma[c], dbeta[c] = the sum of P partial rows, each thread row q of the block
// adding rows q, q + 16, ... and thread row 0 the sixteen sums, in that order.
template <typename T>
__global__ void __launch_bounds__(512)
ln_weight_reduce_kernel(const float *__restrict__ part, int P, int d, int w32, void *dgamma,
                        void *dbeta) {
    __shared__ float sh[16][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * (int64_t)d) {
        const float *p = part + c;
#pragma unroll 10
        for (int k = q; k < P; k += 16) s += p[(int64_t)k * 2 * d];
    }
    sh[q][lane] = s;
    __syncthreads();
    if (q != 0 || c >= 2 * (int64_t)d) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += sh[k][lane];
    void *out = c < d ? dgamma : dbeta;
    if (out == nullptr) return;
    const int64_t i = c < d ? c : c - d;
    if (w32) static_cast<float *>(out)[i] = s;
    else store_f32(static_cast<T *>(out) + i, s);
}

// ---- rows too wide for a ring ------------------------------------------------
//
// Up to 2^31 - 1 elements: vectors are counted in 32 bits without a sign (a thread's step
// past the last one stays above it), the two arrays of weight sums in 64.

// Sum over the block, in a fixed order.
__device__ __forceinline__ float block_sum(float v, float *sh) {
    v = warp_sum(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    return warp_sum(lane < (int)(blockDim.x >> 5) ? sh[lane] : 0.f);
}

template <typename T, int V>
__global__ void __launch_bounds__(1024) ln_forward_wide_kernel(const LnArgs a) {
    __shared__ float sh[32];
    pdl_wait();
    pdl_trigger();
    const uint32_t nvec = a.d / V;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const Raw<T, V> *xp =
            reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.x) + row * a.ldx);
        Raw<T, V> *yp = reinterpret_cast<Raw<T, V> *>(static_cast<T *>(a.y) + row * a.ldy);
        float s = 0.f, f[V];
        for (uint32_t v = threadIdx.x; v < nvec; v += blockDim.x) {
            to_f32<T, V>(xp[v], f);
#pragma unroll
            for (int j = 0; j < V; ++j) s += f[j];
        }
        const float mean = block_sum(s, sh) / (float)a.d;
        s = 0.f;
        for (uint32_t v = threadIdx.x; v < nvec; v += blockDim.x) {
            to_f32<T, V>(xp[v], f);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(f[j] - mean, f[j] - mean, s);
        }
        const float rstd = __frsqrt_rn(block_sum(s, sh) / (float)a.d + a.eps);
        for (uint32_t v = threadIdx.x; v < nvec; v += blockDim.x) {
            to_f32<T, V>(xp[v], f);
#pragma unroll
            for (int j = 0; j < V; ++j)
                f[j] = fmaf((f[j] - mean) * rstd, load_w<T>(a.gamma, a.w32, v * V + j, 1.f),
                            load_w<T>(a.beta, a.w32, v * V + j, 0.f));
            yp[v] = from_f32<T, V>(f);
        }
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(1024) ln_backward_wide_kernel(const LnArgs a) {
    __shared__ float sh[32];
    pdl_wait();
    pdl_trigger();
    const uint32_t nvec = a.d / V;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const Raw<T, V> *xp =
            reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.x) + row * a.ldx);
        const Raw<T, V> *yp =
            reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.dy) + row * a.lddy);
        const Raw<T, V> *rp =
            reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.dres) + row * a.lddres);
        Raw<T, V> *op = reinterpret_cast<Raw<T, V> *>(static_cast<T *>(a.dx) + row * a.lddx);
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.f, s2 = 0.f, x[V], g[V];
        for (uint32_t v = threadIdx.x; v < nvec; v += blockDim.x) {
            to_f32<T, V>(xp[v], x);
            to_f32<T, V>(yp[v], g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gj = g[j] * load_w<T>(a.gamma, a.w32, v * V + j, 1.f);
                s2 += gj;
                s1 = fmaf(gj, (x[j] - mean) * rstd, s1);
            }
        }
        const float c1 = block_sum(s1, sh) / (float)a.d;
        const float c2 = block_sum(s2, sh) / (float)a.d;
        for (uint32_t v = threadIdx.x; v < nvec; v += blockDim.x) {
            to_f32<T, V>(xp[v], x);
            to_f32<T, V>(yp[v], g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float gj = g[j] * load_w<T>(a.gamma, a.w32, v * V + j, 1.f);
                x[j] = rstd * (fmaf(-c1, (x[j] - mean) * rstd, gj) - c2);
            }
            if (a.dres != nullptr) {
                to_f32<T, V>(rp[v], g);
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] += g[j];
            }
            op[v] = from_f32<T, V>(x);
        }
    }
}

// Partial weight gradients of a wide row: a thread per V columns, block row
// blockIdx.y adding rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename T, int V>
__global__ void __launch_bounds__(256) ln_weight_wide_kernel(const LnArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint32_t v = blockIdx.x * 256 + threadIdx.x;
    if (v >= (uint32_t)(a.d / V)) return;
    float dg[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dg[j] = db[j] = 0.f;
    for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
        float x[V], g[V];
        to_f32<T, V>(reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.x) + row * a.ldx)[v], x);
        to_f32<T, V>(reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(a.dy) + row * a.lddy)[v], g);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            db[j] += g[j];
            dg[j] = fmaf(g[j], (x[j] - mean) * rstd, dg[j]);
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.d + (int64_t)v * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        part[j] = dg[j];
        part[a.d + (int64_t)j] = db[j];
    }
}

// ------------------------------------------------------------ host side --

// Vector length (elements) that divides d and every row stride and suits the
// pointers' alignment.
struct Align {
    uint64_t bits = 0;
    void add(const void *p, int64_t ld, int d, int esize, int64_t T) {
        if (p == nullptr) return;
        bits |= reinterpret_cast<uintptr_t>(p) | (uint64_t)d * esize;
        if (T > 1) bits |= (uint64_t)ld * esize;
    }
    bool fits(int bytes) const { return (bits & (bytes - 1)) == 0; }
};

int row_groups(int wpr, int threads) { return std::max(1, threads / (32 * wpr)); }

// Row groups and ring stages of a block of at most max_threads threads (one block
// per SM), with at most T / SMs rounded up groups so that few rows spread over the
// SMs. False where `least` stages of one group do not fit the shared memory. (SHIFT fetches
// a group's next row as soon as all of its threads are done with the last, so one stage
// will do, and more groups with one beat fewer with two: 8192 x 7167 bf16, one group with
// two stages against two with one, backward 174 / 141 us; three against four groups,
// forward 69 / 65. Otherwise a stage is free only at the next row's barrier.)
constexpr size_t kRingSmem = 224 * 1024;
// `fixed` bytes a block, `extra` a group, `stage` a stage.
bool ring_shape(LnArgs &a, int per_thread, int max_threads, size_t fixed, size_t extra, size_t stage,
                int least, int *groups) {
    if (a.d > max_threads * per_thread) return false;
    a.wpr = (a.d + per_thread * 32 - 1) / (per_thread * 32);
    int g = std::min(row_groups(a.wpr, max_threads), a.wpr > 1 ? 15 : kMaxGroups);
    g = (int)std::min<int64_t>(g, std::max<int64_t>(1, (a.T + sm_count() - 1) / sm_count()));
    while (g > 1 && fixed + g * (extra + least * stage) > kRingSmem) --g;
    if (fixed + g * (extra + least * stage) > kRingSmem) return false;
    a.stages = (int)std::min<size_t>(((kRingSmem - fixed) / g - extra) / stage, kRingStages);
    *groups = g;
    return true;
}

// Bytes of the fp32 planes of one weight vector.
template <int V>
size_t plane_bytes(int d) { return ((size_t)d + V - 1) / V * V * sizeof(float); }

template <typename T, int V, int NV, bool SHIFT>
cudaError_t forward_ring(LnArgs a, bool *fits, cudaStream_t s) {
    int groups;
    const size_t stage = SHIFT ? image_bytes(a.d, sizeof(T)) : (size_t)a.d * sizeof(T);
    const size_t fixed = kRingCtl + 2 * plane_bytes<V>(a.d);
    *fits = ring_shape(a, V * NV, kFwdThreads, fixed, SHIFT ? stage : 0, stage, SHIFT ? 1 : 2, &groups);
    if (!*fits) return cudaSuccess;
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(ln_forward_ring_kernel<T, V, NV, SHIFT>), (int)kRingSmem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>((a.T + groups - 1) / groups, sm_count());
    return launch_k(ln_forward_ring_kernel<T, V, NV, SHIFT>, dim3(grid), dim3(groups * a.wpr * 32),
                    fixed + groups * (a.stages + SHIFT) * stage, s, a);
}

template <typename T, int V, int NV, bool SHIFT>
cudaError_t backward_ring(LnArgs a, int *P, bool *fits, cudaStream_t s) {
    int groups;
    const size_t row = SHIFT ? image_bytes(a.d, sizeof(T)) : (size_t)a.d * sizeof(T);
    const size_t stage = row * (a.dres != nullptr ? 3 : 2), fixed = kRingCtl + plane_bytes<V>(a.d);
    // (a group's ring holds its [2][d] fp32 sums in the end)
    const int least = SHIFT && stage + row >= 2 * plane_bytes<V>(a.d) ? 1 : 2;
    *fits = ring_shape(a, V * NV, kBwdRingThreads, fixed, SHIFT ? row : 0, stage, least, &groups);
    if (!*fits) return cudaSuccess;
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(ln_backward_ring_kernel<T, V, NV, SHIFT>), (int)kRingSmem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>((a.T + groups - 1) / groups, std::min(sm_count(), kLnPartials));
    *P = grid;
    return launch_k(ln_backward_ring_kernel<T, V, NV, SHIFT>, dim3(grid), dim3(groups * a.wpr * 32),
                    fixed + groups * (a.stages * stage + SHIFT * row), s, a);
}

// Vectors a thread: one or two where a warp still holds the row, else four.
template <typename T, bool SHIFT>
cudaError_t forward_rows(const LnArgs &a, bool *fits, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if (a.d <= 32 * W) return forward_ring<T, W, 1, SHIFT>(a, fits, s);
    if (a.d <= 64 * W) return forward_ring<T, W, 2, SHIFT>(a, fits, s);
    return forward_ring<T, W, 4, SHIFT>(a, fits, s);
}
template <typename T, bool SHIFT>
cudaError_t backward_rows(const LnArgs &a, int *P, bool *fits, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if (a.d <= 32 * W) return backward_ring<T, W, 1, SHIFT>(a, P, fits, s);
    if (a.d <= 64 * W) return backward_ring<T, W, 2, SHIFT>(a, P, fits, s);
    return backward_ring<T, W, 4, SHIFT>(a, P, fits, s);
}

template <typename T>
cudaError_t forward_type(const LnArgs &a, const Align &al, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);  // elements of a 16-byte vector
    bool fits = false;
    const cudaError_t e =
        al.fits(16) ? forward_rows<T, false>(a, &fits, s) : forward_rows<T, true>(a, &fits, s);
    if (e != cudaSuccess || fits) return e;
    const int grid = (int)std::min<int64_t>(a.T, 2 * sm_count());
    return al.fits(16) ? launch_k(ln_forward_wide_kernel<T, W>, dim3(grid), dim3(1024), 0, s, a)
                       : launch_k(ln_forward_wide_kernel<T, 1>, dim3(grid), dim3(1024), 0, s, a);
}

template <typename T>
cudaError_t backward_type(const LnArgs &a, const Align &al, void *dgamma, void *dbeta,
                          cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    int P = 0;
    bool fits = false;
    cudaError_t e =
        al.fits(16) ? backward_rows<T, false>(a, &P, &fits, s) : backward_rows<T, true>(a, &P, &fits, s);
    if (e != cudaSuccess) return e;
    if (!fits) {
        // the weights' sums first: dx may be written over dy
        const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(a.T, 2 * sm_count()));
        if (a.part != nullptr) {
            P = ln_partials(a.T);
            const int v = al.fits(16) ? W : 1;
            const dim3 g((a.d / v + 255u) / 256, P);
            e = al.fits(16) ? launch_k(ln_weight_wide_kernel<T, W>, g, dim3(256), 0, s, a)
                            : launch_k(ln_weight_wide_kernel<T, 1>, g, dim3(256), 0, s, a);
            if (e != cudaSuccess) return e;
        }
        e = al.fits(16) ? launch_k(ln_backward_wide_kernel<T, W>, dim3(grid), dim3(1024), 0, s, a)
                        : launch_k(ln_backward_wide_kernel<T, 1>, dim3(grid), dim3(1024), 0, s, a);
    }
    if (e != cudaSuccess || a.part == nullptr) return e;
    return launch_k(ln_weight_reduce_kernel<T>, dim3((unsigned)((2ll * a.d + 31) / 32)), dim3(512), 0, s,
                    static_cast<const float *>(a.part), P, a.d, a.w32, dgamma, dbeta);
}

}  // namespace

int ln_partials(int64_t T) { return (int)std::max<int64_t>(1, std::min<int64_t>(T, kLnPartials)); }

cudaError_t launch_layernorm_forward(const void *x, int64_t ldx, const void *gamma, const void *beta,
                                     void *y, int64_t ldy, float *mean, float *rstd, int64_t T,
                                     int d, float eps, moe_dtype_t type, bool w32, int64_t withheld,
                                     cudaStream_t s) {
    LnArgs a{};
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldy = ldy;
    a.T = T;
    a.d = d;
    a.w32 = w32;
    a.withheld = withheld;
    a.eps = eps;
    const int es = type == MOE_DTYPE_F32 ? 4 : 2;
    Align al;
    al.add(x, ldx, d, es, T);
    al.add(y, ldy, d, es, T);
    switch (type) {
        case MOE_DTYPE_BF16: return forward_type<__nv_bfloat16>(a, al, s);
        case MOE_DTYPE_F16: return forward_type<__half>(a, al, s);
        default: return forward_type<float>(a, al, s);
    }
}

cudaError_t launch_layernorm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                      const void *gamma, const float *mean, const float *rstd,
                                      const void *dres, int64_t lddres, void *dx, int64_t lddx,
                                      void *dgamma, void *dbeta, int64_t T, int d,
                                      moe_dtype_t type, bool w32, float *part, int64_t withheld,
                                      cudaStream_t s) {
    LnArgs a{};
    a.x = x;
    a.gamma = gamma;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dy = dy;
    a.dres = dres;
    a.dx = dx;
    a.ldx = ldx;
    a.lddy = lddy;
    a.lddres = lddres;
    a.lddx = lddx;
    a.T = T;
    a.d = d;
    a.w32 = w32;
    a.withheld = withheld;
    a.part = dgamma != nullptr || dbeta != nullptr ? part : nullptr;
    const int es = type == MOE_DTYPE_F32 ? 4 : 2;
    Align al;
    al.add(dy, lddy, d, es, T);
    al.add(x, ldx, d, es, T);
    al.add(dres, lddres, d, es, T);
    al.add(dx, lddx, d, es, T);
    switch (type) {
        case MOE_DTYPE_BF16: return backward_type<__nv_bfloat16>(a, al, dgamma, dbeta, s);
        case MOE_DTYPE_F16: return backward_type<__half>(a, al, dgamma, dbeta, s);
        default: return backward_type<float>(a, al, dgamma, dbeta, s);
    }
}

}  // namespace moe
