// Dense gated feed-forward block for few tokens (decoding): the weights are
// streamed once and nothing else is large, so HBM bounds it: 2 d n weights for
// H = act(X W1) * (X W3), d n for Y = H W2.
//
// The tensor cores take the weights as the 128-row operand: a tile is 128 columns
// of W (TMA boxes of 64 columns x 64 rows, MN-major) against NT tokens (16 .. 128,
// padded with zeros by TMA), so the accumulator holds the transposed output, one
// weight column per TMEM lane and one token per TMEM column, and one token costs
// no more MMA time than its share of the weight traffic.
//
// All tiles' k-blocks (64 rows of W) form one sequence, cut into equal runs, one
// per CTA, whatever the number of tiles: every SM reads the same number of bytes.
// A tile that is cut is joined by its parts: each warp writes its part (fp32) to
// the workspace and takes a ticket; the last to arrive adds all parts in the order
// of the runs (so the result does not depend on who is last), applies the
// activation and stores. Nobody waits. Tickets return to zero with the last
// arrival.
//
// The second product is launched to overlap the first (programmatic dependent
// launch): its CTAs fill their weight stages, which do not depend on H, and only
// then wait for the first kernel. Both kernels' shared memory and TMEM fit one SM
// together for up to 32 tokens.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2 TMEM allocation, 4-7 epilogue.
#include <algorithm>

#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int BK = 64;
constexpr uint32_t kBox = 64 * 64 * 2;  // 8 KB: 64 columns x 64 rows of W
constexpr uint32_t kMat = 2 * kBox;     // 128 columns
constexpr int kMaxStages = 8;

// MATS weight matrices (2: gate and up; 1: down), NT tokens.
template <int MATS, int NT>
struct Geo {
    static constexpr uint32_t kTok = NT * BK * 2;
    static constexpr uint32_t kStageBytes = MATS * kMat + kTok;
    // half an SM's shared memory for up to 32 tokens, else all of it
    static constexpr uint32_t kBudget = NT <= 32 ? 108 * 1024 : 216 * 1024;
    static constexpr int kStages =
        kBudget / kStageBytes < kMaxStages ? kBudget / kStageBytes : kMaxStages;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
    // two accumulators of MATS * NT columns
    static constexpr uint32_t kTmem = 2 * MATS * NT < 32 ? 32 : 2 * MATS * NT;
};

struct SmallMaps {
    CUtensorMap w[2], x;
};

struct SmallArgs {
    int T, cols;   // tokens, output columns
    int kbs;       // k-blocks per tile
    int tiles;
    int act, f16;
    uint32_t idesc;
    int early;     // weights may be read before the previous kernel has finished
    void *out;     // [T, cols], 16 bits
    float *part;   // [CTA][2][MATS][T][128]
    uint32_t *ticket;  // [tiles][4]
    uint32_t *err;
};

struct SmallCtl {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
};
static_assert(sizeof(SmallCtl) <= 256, "control block");

// First k-block of CTA c's run among W of them.
__device__ __forceinline__ int64_t run_start(int64_t W, int c) { return W * c / (int)gridDim.x; }

// TMEM: 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <int MATS, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 32 ? 2 : 1)
stream_gemm_kernel(const __grid_constant__ SmallMaps maps, const SmallArgs args) {
    using G = Geo<MATS, NT>;
    constexpr int S = G::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    SmallCtl *ctl = reinterpret_cast<SmallCtl *>(smem + (size_t)S * G::kStageBytes);
    const uint32_t base = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&ctl->tfull[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->tempty[a]), 4);
        }
        ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
        ptx::fence_barrier_init();
    }
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), G::kTmem);
        ptx::tmem_relinquish();
    }
    if (!args.early) {
        pdl_wait();
        pdl_trigger();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;

    const int64_t W = (int64_t)args.tiles * args.kbs;
    const int64_t begin = run_start(W, blockIdx.x), end = run_start(W, blockIdx.x + 1);
    const int count = (int)(end - begin);

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------ producer --
        auto load_w = [&](int64_t i, uint32_t s) {
            const int tile = (int)(i / args.kbs), kb = (int)(i - (int64_t)tile * args.kbs);
            const uint32_t full = ptx::smem_addr(&ctl->full[s]), dst = base + s * G::kStageBytes;
            ptx::mbar_arrive_expect_tx(full, G::kStageBytes);
#pragma unroll
            for (int m = 0; m < MATS; ++m) {
                ptx::tma_load_2d(dst + m * kMat, &maps.w[m], full, tile * 128, kb * BK);
                ptx::tma_load_2d(dst + m * kMat + kBox, &maps.w[m], full, tile * 128 + 64, kb * BK);
            }
        };
        auto load_x = [&](int64_t i, uint32_t s) {
            const int kb = (int)(i % args.kbs);
            ptx::tma_load_2d(base + s * G::kStageBytes + MATS * kMat, &maps.x,
                             ptx::smem_addr(&ctl->full[s]), kb * BK, 0);
        };
        int it = 0;
        bool ok = true;
        if (args.early) {
            // the stages' weights, then (once the previous kernel has finished) its output
            const int ahead = min(count, S);
            for (int j = 0; j < ahead; ++j) load_w(begin + j, j);
            pdl_wait();
            ptx::fence_proxy_async_global();
            for (int j = 0; j < ahead; ++j) load_x(begin + j, j);
            it = ahead;
        }
        for (; it < count; ++it) {
            const uint32_t s = it % S;
            if (!bounded_wait(ptx::smem_addr(&ctl->empty[s]), ((it / S) & 1u) ^ 1u, args.err)) {
                ok = false;
                break;
            }
            load_w(begin + it, s);
            load_x(begin + it, s);
        }
        if (!ok)
            for (int j = max(0, it - S); j < it; ++j)
                bounded_wait(ptx::smem_addr(&ctl->full[j % S]), (j / S) & 1u, args.err);
    } else if (warp == 1 && lane == 0) {
        // ---------------------------------------------------- MMA issuer --
        int seg = -1;
        int64_t seg_tile = -1;
        bool ok = true;
        for (int it = 0; it < count; ++it) {
            const int64_t tile = (begin + it) / args.kbs;
            const bool first = tile != seg_tile;
            if (first) {
                if (seg >= 0) ptx::tc_commit(ptx::smem_addr(&ctl->tfull[seg & 1]));
                ++seg;
                seg_tile = tile;
                if (!bounded_wait(ptx::smem_addr(&ctl->tempty[seg & 1]), ((seg >> 1) & 1) ^ 1, args.err)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
            }
            const uint32_t s = it % S;
            if (!bounded_wait(ptx::smem_addr(&ctl->full[s]), (it / S) & 1u, args.err)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t sW = base + s * G::kStageBytes, sX = sW + MATS * kMat;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
                const uint64_t bd = ptx::desc_sw128(sX + k * 32, 16, 1024);
#pragma unroll
                for (int m = 0; m < MATS; ++m)
                    ptx::tc_mma_f16(tmem_base + ((seg & 1) * MATS + m) * NT,
                                    ptx::desc_sw128(sW + m * kMat + k * 2048, kBox, 1024), bd,
                                    args.idesc, !first || k != 0);
            }
            ptx::tc_commit(ptx::smem_addr(&ctl->empty[s]));
        }
        if (ok && seg >= 0) ptx::tc_commit(ptx::smem_addr(&ctl->tfull[seg & 1]));
        ptx::tc_commit(ptx::smem_addr(&ctl->drain));
        bounded_wait(ptx::smem_addr(&ctl->drain), 0, args.err);
    } else if (warp >= 4) {
        // ------------------------------------------------------ epilogue --
        const int q = warp & 3, T = args.T;
        const bool f16 = args.f16 != 0;
        uint16_t *out = static_cast<uint16_t *>(args.out);
        if (args.early) pdl_wait();  // the previous kernel's tickets and parts, and H's readers
        const int64_t part_ld = (int64_t)MATS * T * 128;  // floats of one part
        int64_t i = begin;
        for (int seg = 0; i < end; ++seg) {
            const int tile = (int)(i / args.kbs);
            const int64_t t0 = (int64_t)tile * args.kbs, t1 = t0 + args.kbs;
            const bool whole = i == t0 && end >= t1;
            const int a = seg & 1;
            if (!bounded_wait(ptx::smem_addr(&ctl->tfull[a]), (seg >> 1) & 1, args.err)) break;
            ptx::tc_fence_after();
            const uint32_t taddr =
                tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * MATS * NT;
            const int col = tile * 128 + q * 32 + lane;
            // the result of one token from its sums
            auto emit = [&](int t, float s0, float s1) {
                const float v = MATS == 2 ? s0 * act_sigmoid(s0, args.act) * s1 : s0;
                if (col < args.cols) out[(int64_t)t * args.cols + col] = round16(v, f16);
            };
            // part of CTA c for this tile: a run's first tile goes to slot 0, a
            // later one (its last) to slot 1
            auto slot = [&](int c) {
                const int64_t b = run_start(W, c);
                return args.part + ((int64_t)c * 2 + (b / args.kbs == tile ? 0 : 1)) * part_ld +
                       q * 32 + lane;
            };
            float *mine = whole ? nullptr : slot(blockIdx.x);
#pragma unroll 1
            for (int c = 0; c < NT && c < T; c += 16) {
                uint32_t r[MATS][16];
#pragma unroll
                for (int m = 0; m < MATS; ++m) tmem_ld16(taddr + m * NT + c, r[m]);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (c + j >= T) break;
                    if (whole) {
                        emit(c + j, __uint_as_float(r[0][j]), __uint_as_float(r[MATS - 1][j]));
                    } else {
#pragma unroll
                        for (int m = 0; m < MATS; ++m)
                            __stcg(mine + (int64_t)(m * T + c + j) * 128, __uint_as_float(r[m][j]));
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->tempty[a]));
            if (!whole) {
                // the runs that hold k-blocks of this tile
                int c0 = (int)(t0 * (int)gridDim.x / W), c1;
                while (run_start(W, c0 + 1) <= t0) ++c0;
                c1 = c0;
                while (run_start(W, c1 + 1) < t1) ++c1;
                __threadfence();
                __syncwarp();
                uint32_t arrived = 0;
                uint32_t *ticket = args.ticket + tile * 4 + q;
                if (lane == 0) arrived = atomicAdd(ticket, 1u);
                arrived = __shfl_sync(0xffffffffu, arrived, 0);
                if (arrived == (uint32_t)(c1 - c0)) {  // the last part
                    __threadfence();
#pragma unroll 1
                    for (int t = 0; t < T; t += 16) {
                        float sum[MATS][16];
#pragma unroll
                        for (int m = 0; m < MATS; ++m)
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[m][j] = 0.f;
#pragma unroll 2
                        for (int c = c0; c <= c1; ++c) {
                            const float *p = slot(c) + (int64_t)t * 128;
#pragma unroll
                            for (int m = 0; m < MATS; ++m)
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (t + j < T) sum[m][j] += __ldcg(p + (int64_t)(m * T + j) * 128);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (t + j < T) emit(t + j, sum[0][j], sum[MATS - 1][j]);
                    }
                    if (lane == 0) *ticket = 0;
                }
            }
            i = min(end, t1);
        }
    }
    // the next kernel may start its own loads once this one is past its main loop
    if (args.early) {
        if (warp != 0 && warp < 4) pdl_wait();
        pdl_trigger();
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc(tmem_base, G::kTmem);
}

template <int MATS, int NT>
cudaError_t launch_nt(const SmallMaps &maps, SmallArgs args, int grid, cudaStream_t s) {
    constexpr size_t kSmem = Geo<MATS, NT>::kSmem;
    args.idesc = idesc(args.f16 != 0, 128, NT, true, false);
    const cudaError_t e = ensure_dynamic_smem(
        reinterpret_cast<const void *>(stream_gemm_kernel<MATS, NT>), (int)kSmem);
    if (e != cudaSuccess) return e;
    return launch_k(stream_gemm_kernel<MATS, NT>, dim3(grid), dim3(kThreads), kSmem, s, maps, args);
}

int padded_tokens(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

// CTAs of one product: one per SM, fewer where a run would be under four k-blocks
// (then the joining costs more than the shorter runs save).
int stream_grid(int cols, int K, int sms) {
    const int64_t tiles = (cols + 127) / 128, W = tiles * ((K + BK - 1) / BK);
    return (int)std::min<int64_t>(std::min(sms, kFfnMaxCtas), std::max(tiles, W / 4));
}

cudaError_t launch_stream(int mats, const void *w0, const void *w1, const void *x, int T, int K,
                          int cols, int act, bool f16, bool early, void *out, float *part,
                          uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    const int nt = padded_tokens(T);
    SmallMaps m{};
    const CUtensorMapDataType ty = map_type(f16);
    if (!make_map(&m.w[0], ty, w0, cols, K, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&m.w[1], ty, w1, cols, K, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&m.x, ty, x, K, T, 64, nt, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    SmallArgs a{};
    a.T = T;
    a.cols = cols;
    a.kbs = (K + BK - 1) / BK;
    a.tiles = (cols + 127) / 128;
    a.act = act;
    a.f16 = f16;
    a.early = early;
    a.out = out;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    const int grid = stream_grid(cols, K, sm_count());
#define MOE_CASE(N)                                                      \
    case N:                                                              \
        return mats == 2 ? launch_nt<2, N>(m, a, grid, s) : launch_nt<1, N>(m, a, grid, s)
    switch (nt) {
        MOE_CASE(16);
        MOE_CASE(32);
        MOE_CASE(64);
        default:
            MOE_CASE(128);
    }
#undef MOE_CASE
}

}  // namespace
}  // namespace ffn

using namespace ffn;

size_t ffn_stream_part_bytes(int T, int d, int n) {
    // two parts for each CTA, of two matrices in the first product
    const size_t ctas = std::max(2 * stream_grid(n, d, kFfnMaxCtas), stream_grid(d, n, kFfnMaxCtas));
    return ctas * 2 * T * 128 * sizeof(float);
}

cudaError_t launch_ffn_stream(const void *X, const void *W1, const void *W3, const void *W2, int T,
                              int d, int n, int act, bool f16, void *H, void *Y, float *part,
                              uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    cudaError_t e = launch_stream(2, W1, W3, X, T, d, n, act, f16, false, H, part, ticket, err, s);
    if (e != cudaSuccess) return e;
    // the second product touches the parts and tickets only after the first is done
    return launch_stream(1, W2, W2, H, T, n, d, act, f16, true, Y, part, ticket, err, s);
}

}  // namespace moe
