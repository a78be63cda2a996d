// The norms around a block in one pass over the stream (block_norm_forward.cuh, its gradients in
// block_norm_backward.cuh). For a row of d elements,
//   bh = b r_post,  r_post = 1 / sqrt(mean(b^2) + eps)   (1 without the post norm)
//   n  = post bh
//   y  = scale x + g n,   g = sigmoid(gate) of the row or the element, or 1
//   yh = y r_pre,   r_pre = 1 / sqrt(mean(y^2) + eps),   u = pre yh
// y is rounded for the output alone: u is that of the fp32 y. Without a block (b NULL) y = x
// and only u is written: a plain RMS norm.
#pragma once

#include <algorithm>

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
    uint32_t group_bytes;  // of a row group's ring
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

// The same over the warps of a row group of both CTAs of a pair, which hold half of the row each: a
// warp gives its value to both CTAs and arrives on both barriers (of 2 wpr arrivals), two of
// each in turn. A wait that runs out (after the limits of the waits for rows, which the other
// CTA may be in: its device has stopped) gives NaN, and no later one waits.
struct PairCtl {
    uint64_t bar[16][2];
    float slots[16][2][32];
};
struct PairSum {
    PairCtl *ctl;
    int group, wg, wpr;
    uint32_t rank;
    int count = 0;
    bool dead = false;
    __device__ __forceinline__ float operator()(float v) {
        const int lane = threadIdx.x & 31, k = count & 1;
        const uint32_t parity = (count >> 1) & 1;
        ++count;
        // (a warp that no longer waits may arrive early: with NaN, so that no sum it is in has a value)
        v = warp_sum(dead ? NAN : v);
        const uint32_t bar = ptx::smem_addr(&ctl->bar[group][k]);
        if (lane < 2) {
            const uint32_t to = ptx::smem_addr(&ctl->slots[group][k][rank * wpr + wg]);
            ptx::st_cluster_f32(ptx::mapa(to, lane), v);
            ptx::mbar_arrive_cluster(ptx::mapa(bar, lane));
        }
        if (!dead && !ptx::mbar_try_wait_cluster(bar, parity)) dead = !wait_long(bar, parity);
        if (dead) return NAN;
        return warp_sum(lane < 2 * wpr ? ctl->slots[group][k][lane] : 0.f);
    }
    static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
        const uint64_t t0 = ptx::globaltimer_ns();
        for (;;) {
            const bool late = ptx::globaltimer_ns() - t0 > 4 * kWaitLimitNs;
            if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
            if (late) return false;
        }
    }
};

// Packed sigmoid g of z, and h = 1 - g, for 16-bit results: with t = 2^(-z log2 e), g = 1 / (1 + t)
// and h = t g, which does not cancel. (t infinite: g is 0, and the minimum with 1 takes the
// place of infinity times 0. Where 1 + t is past 2^126, z < -87.3, g is 0.) The exponent's own
// rounding shows as |z| 2^-24 of the smaller of the two.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <typename T, bool WANT_H>
__device__ __forceinline__ void sigmoid2(f32x2 z, f32x2 &g, f32x2 &h) {
    float a, b, ga, gb, ha, hb;
    if constexpr (sizeof(T) == 4) {
        unpair(z, a, b);
        sigmoid(a, ga, ha);
        sigmoid(b, gb, hb);
        g = pair(ga, gb);
        if (WANT_H) h = pair(ha, hb);
    } else {
        unpair(mul2(z, both(-1.44269504f)), a, b);
        const f32x2 t = pair(exp2_approx(a), exp2_approx(b));
        unpair(add2(t, both(1.f)), a, b);
        g = pair(rcp_approx(a), rcp_approx(b));
        if (WANT_H) {
            unpair(mul2(t, g), ha, hb);
            h = pair(fminf(ha, 1.f), fminf(hb, 1.f));
        }
    }
}

// ---- rings of rows (as layer norm's, see norm.cu): each row group keeps the rows of its
// operands that come next in stages of shared memory, filled by bulk copies.
//
// SHIFT: rows that start anywhere. They come as images of the 16-byte blocks that hold them,
// and a block of threads takes rows r, r + 8, r + 16, ... only: eight rows on, every row starts
// at the same place of its 16 bytes again, whatever the stride. So a thread's vectors are the
// image's blocks, with the same columns in all of its rows, and nothing is shifted but the
// weights, once; the elements of the first and the last block that are not the row's are set to
// zero. The place is that of the first output's rows; where (SHIFT 2) an operand's rows start
// elsewhere its vectors are shifted out of two neighbouring blocks, and another output's elements
// are stored one by one.
constexpr int kRingStages = 2, kMaxGroups = 28, kPhases = 8;
struct RingCtl {
    uint64_t full[kMaxGroups][kRingStages];
    float slots[2][32];
    float scalars[kMaxGroups][kRingStages][4];  // r_pre, r_post and the gate of a stage's row
};
constexpr size_t kRingCtl = (sizeof(RingCtl) + 127) / 128 * 128;

// Warps a row, row groups and ring stages of a block of at most max_threads, one of `sms`; false
// where a stage of one group does not fit. cols: columns that a row's vectors may reach over; `fixed` bytes
// a block, `stage` a stage, `least` a group's ring (which stages alone may leave smaller).
bool shape_of(Args &a, int cols, int per_thread, int max_threads, int sms, size_t fixed, size_t stage,
              size_t least, int *groups);
// Rows of a block in hand: a group with one stage fetches its next row late, with two it need not.
inline int rows_ahead(const Args &a, int groups) { return groups * std::min(a.stages, 2); }
// Blocks of a launch of rows in `groups` a block.
template <int SHIFT>
int ring_grid(int64_t T, int groups, int sms) {
    if (!SHIFT) return (int)std::min<int64_t>((T + groups - 1) / groups, sms);
    const int64_t of_phase = (T + kPhases - 1) / kPhases;
    return kPhases * (int)std::min<int64_t>((of_phase + groups - 1) / groups, std::max(1, sms / kPhases));
}
// Columns that a row's vectors may reach over; bytes of a row in a stage. (A vector that is
// shifted out of two blocks may reach a block past the image, or lie one in front of it.)
template <int V, int SHIFT>
__host__ __device__ constexpr int ring_cols(int d) { return SHIFT ? d + V - 1 : d; }
template <typename T, int SHIFT>
__host__ __device__ uint32_t ring_row_bytes(int d) {
    return SHIFT ? (image_bytes(d, sizeof(T)) + 16 + 112 + 127) / 128 * 128 : (uint32_t)(d * sizeof(T));
}

// q with zeros for the elements outside [first, end).
template <typename T>
__device__ __forceinline__ uint4 elements_inside(uint4 q, int first, int end) {
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            if (j < first || j >= end) w[j] = 0;
        } else {
            if (2 * j < first || 2 * j >= end) w[j] &= 0xffff0000u;
            if (2 * j + 1 < first || 2 * j + 1 >= end) w[j] &= 0x0000ffffu;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's vectors of V elements of a row: vector v holds the columns v V - lead and on.
template <typename T, int V, int SHIFT>
struct Part {
    int tpr, t, d, nvec;
    int lead;  // elements of the first block in front of the row
    // out: an output's row of this block
    __device__ __forceinline__ Part(int tpr_, int t_, int d_, const void *out) : tpr(tpr_), t(t_), d(d_) {
        lead = SHIFT ? (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T)) : 0;
        nvec = (d + lead + V - 1) / V;
    }
    __device__ __forceinline__ bool has(int i) const { return i * tpr + t < nvec; }
    // a row's start in global memory, against the output's place
    __device__ __forceinline__ int off(const T *row) const {
        return SHIFT == 2 ? (int)(reinterpret_cast<uintptr_t>(row) & 15) - lead * (int)sizeof(T) : 0;
    }
    // vector i of the row at `image`, which starts `off` bytes off that place
    __device__ __forceinline__ void load(const uint8_t *image, int off, int i, f32x2 (&p)[V / 2]) const {
        const int v = i * tpr + t;
        if constexpr (!SHIFT) {
            to_pairs<T, V>(reinterpret_cast<const uint4 *>(image)[v], p);
        } else {
            uint4 q = SHIFT == 1 || off == 0
                               ? reinterpret_cast<const uint4 *>(image)[v]
                               : image_vec<T>(image - (off < 0 ? 16 : 0), v, (uint32_t)off & 15);
            if (v == 0 || v == nvec - 1) q = elements_inside<T>(q, lead - v * V, d + lead - v * V);
            to_pairs<T, V>(q, p);
        }
    }
    // vector i to the row in global memory
    __device__ __forceinline__ void store(T *row, int off, int i, const f32x2 (&p)[V / 2]) const {
        const int v = i * tpr + t;
        const uint4 q = from_pairs<T, V>(p);
        if constexpr (!SHIFT) {
            reinterpret_cast<uint4 *>(row)[v] = q;
        } else if ((SHIFT == 1 || off == 0) && v > 0 && v < nvec - 1) {
            *reinterpret_cast<uint4 *>(row + (v * V - lead)) = q;
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = v * V - lead + j;
                if (c < 0 || c >= d) continue;
                if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(row)[c] = w[j];
                else reinterpret_cast<uint16_t *>(row)[c] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
};
// A weight vector in shared memory, `lead` elements on: in fp32 as planes of four elements of
// every vector, or (RAW) of 16 bits as it is. Both are read without bank conflicts; planes need
// no conversion, RAW half the memory.
template <typename T, int V, int SHIFT, bool RAW>
struct Weights {
    static __host__ __device__ uint32_t bytes(int d) {
        const uint32_t n = (uint32_t)((ring_cols<V, SHIFT>(d) + V - 1) / V * V) * (RAW ? sizeof(T) : sizeof(float));
        return SHIFT ? (n + 127) / 128 * 128 : n;
    }
    // (first: the column that the part starts with)
    static __device__ __forceinline__ void fill(uint8_t *to, const void *w, int w32, const Part<T, V, SHIFT> &part,
                                                int first = 0) {
        for (int v = threadIdx.x; v < part.nvec; v += blockDim.x) {
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = v * V + j - part.lead;
                f[j] = c >= 0 && c < part.d ? load_w<T>(w, w32, first + c, 1.f) : 0.f;
            }
            if constexpr (RAW) {
                reinterpret_cast<uint4 *>(to)[v] = from_f32<T, V>(f);
            } else {
#pragma unroll
                for (int h = 0; h < V / 4; ++h)
                    reinterpret_cast<float4 *>(to)[h * part.nvec + v] =
                        make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
            }
        }
    }
    static __device__ __forceinline__ void load(const Part<T, V, SHIFT> &part, const uint8_t *w, int i, f32x2 (&g)[V / 2]) {
        const int v = i * part.tpr + part.t;
        if constexpr (RAW) to_pairs<T, V>(reinterpret_cast<const uint4 *>(w)[v], g);
        else plane_pairs<V>(reinterpret_cast<const float *>(w), part.nvec, v, g);
    }
};
// Where the image of a row lies in its place of a stage: as far from a 128-byte line of shared
// memory as the row is from one of global memory, so that a bulk copy moves whole lines.
template <typename T, int SHIFT>
__device__ __forceinline__ uint32_t image_at(const void *p, int64_t ld, int64_t r) {
    return SHIFT ? (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const T *>(p) + r * ld) & 112 : 0;
}
// One thread: row r of a [rows, d] tensor into dst, arriving on bar.
template <typename T, int SHIFT>
__device__ __forceinline__ void fetch_row(uint8_t *dst, const void *p, int64_t ld, int64_t r, int64_t rows, int d,
                                          uint32_t bar) {
    const T *base = static_cast<const T *>(p);
    if constexpr (SHIFT) {
        ptx::mbar_arrive_expect_tx(bar, fetch_image(dst + image_at<T, SHIFT>(p, ld, r), base, ld, r, rows, d, bar));
    } else {
        ptx::mbar_arrive_expect_tx(bar, (uint32_t)(d * sizeof(T)));
        ptx::bulk_load(ptx::smem_addr(dst), base + r * ld, (uint32_t)(d * sizeof(T)), bar);
    }
}

// One thread: a row's scalars (those that there are), arriving on bar when they are there. They come
// with the row, as a load at its start is waited for there (8192 x 7168 bf16 with a row's gate,
// forward 82 / 77 us, backward 186 / 136; 4096 x 4096, 27 / 24.4 and 58 / 45).
__device__ __forceinline__ void fetch_scalars(float *to, const float *r_pre, const float *r_post, const float *gate,
                                              int64_t r, uint32_t bar) {
    const uint32_t dst = ptx::smem_addr(to);
    if (r_pre != nullptr) ptx::cp_async_4(dst, r_pre + r);
    if (r_post != nullptr) ptx::cp_async_4(dst + 4, r_post + r);
    if (gate != nullptr) ptx::cp_async_4(dst + 8, gate + r);
    ptx::cp_async_arrive(bar);
}

// Threads of a block without a ring, its row groups, and its grid.
constexpr int kRowThreads = 512;
struct RowShape {
    int groups, grid;
};
RowShape row_shape(Args &a, int per_thread);

// How the rows of a call's matrices start: 0 all on 16 bytes, 1 all at the same places, 2 anywhere.
struct Places {
    Align al;
    uint64_t first = 0, other = 0;
    bool any = false;
    void add(const void *p, int64_t ld, int d, int esize, int64_t T) {
        if (p == nullptr) return;
        al.add(p, ld, d, esize, T);
        const uint64_t at = (reinterpret_cast<uintptr_t>(p) & 15) | (T > 1 ? ((uint64_t)ld * esize & 15) << 4 : 0);
        if (!any) first = at;
        any = true;
        other |= at ^ first;
    }
    int shift() const { return al.fits(16) ? 0 : other == 0 ? 1 : 2; }
};

// The launches for one element type (block_norm_*.cu).
template <typename T>
cudaError_t forward_type(const Args &a, int shift, cudaStream_t s);
template <typename T>
cudaError_t backward_type(const Args &a, int shift, int *P, cudaStream_t s);

}  // namespace bn
}  // namespace moe
