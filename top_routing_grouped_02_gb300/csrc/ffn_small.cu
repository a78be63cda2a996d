// Dense gated feed-forward block for few tokens (decoding), one persistent launch:
//   H = act(X W1) * (X W3), Y = H W2.
// The weights are streamed once and nothing else is large, so HBM bounds it.
//
// The tensor cores take the weights as the 128-row operand: a tile is 128 columns
// of W (TMA boxes of 64 columns x 64 rows, MN-major) against NT tokens (16 .. 64,
// padded with zeros by TMA), so the accumulator holds the transposed output, one
// weight column per TMEM lane and one token per TMEM column, and one token costs
// no more MMA time than its share of the weight traffic.
//
// Each product is a sequence of units of 32 KB of weights (gate and up: 64 rows of
// both matrices; down: 128 rows), cut into equal runs, one per CTA and SM,
// whatever the number of tiles: every SM reads the same number of bytes. A tile
// that is cut is joined by the CTAs that hold its parts: each writes its part (fp32)
// to the workspace, and once all have, each adds all parts of its share of the
// tokens, in the order of the runs, so the result does not depend on timing.
//
// The down projection needs all of H: a grid-wide counter separates the products.
// The rings of all SMs (about 200 KB each) meanwhile fill with W2, which does not
// depend on H, and once most CTAs are through with the first product, L2 fills with
// more of it, so HBM stays busy through the joins and the barrier. All CTAs are
// resident together (one per SM); every wait is bounded. The counters return to
// zero with the launch.
//
// Measured: one token, d = 4096, n = 14336 bf16 63.4 us (5.6 TB/s; a kernel that only loads
// as much reaches 6.05); 48 tokens, 7168 x 2048 fp16 31.6 us, of which the loads need 15:
// the first product's last sums are in the workspace at 16 us, H is complete at 19.5, the
// second product's sums at 25 and joined at 29.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2 TMEM allocation, 4-11 epilogue.
#include <algorithm>

#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace {

// Epilogue warpgroups: they share the columns of a dump and the vectors of a join (48
// tokens, d = 7168, n = 2048: one 32.9 us, two 32.2 us, three 32.3 us).
constexpr int kSets = 2;
constexpr int kThreads = 128 + 128 * kSets;
constexpr int BK = 64;
constexpr uint32_t kBox = 64 * 64 * 2;    // 8 KB: 64 columns x 64 rows of W
constexpr uint32_t kMat = 2 * kBox;       // 128 columns
constexpr uint32_t kWBytes = 2 * kMat;    // weights of one unit
constexpr int kMaxStages = 6;
// CTAs (in eighths) that have their part of H before W2 is fetched into L2 beyond the
// rings, and how many units of it (one token, d = 4096, n = 14336: none 65.3 us, 8 units
// 64.2, 12 or 16 63.4; the same 12 at six eighths 63.5, 8 at five eighths 64.5).
constexpr int kAheadNum = 7, kAheadUnits = 12;
// control words (behind the error word): grid arrivals, exits
constexpr int kWordGrid = 8, kWordExit = 9;

template <int NT>
struct Geo {
    static constexpr uint32_t kTok = NT * BK * 2;  // 64 of the reduction of all tokens
    static constexpr uint32_t kStageBytes = kWBytes + 2 * kTok;
    static constexpr int kStages = std::min<int>(kMaxStages, 216 * 1024 / kStageBytes);
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
    static constexpr uint32_t kTmem = 4 * NT;  // two accumulators of two matrices
};

// One product: out[T, cols] from the reduction over K.
struct Product {
    int cols, K, kbs, tiles, ctas;  // kbs: units per tile
    void *out;
};

struct SmallMaps {
    CUtensorMap w[3], x, h;
};

struct SmallArgs {
    Product p[2];
    int T, act, f16;
    uint32_t idesc;
    float *part;       // [CTA][2][matrices][T / 4][128][4]
    uint32_t *ticket;  // [tiles of both products][4]
    uint32_t *err;
};

struct SmallCtl {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
};
static_assert(sizeof(SmallCtl) <= 256, "control block");

// The units of a product cut into equal runs, one per CTA, whatever the tiles they
// belong to.
struct Runs {
    int64_t W;
    int parts;
    __device__ __forceinline__ Runs(const Product &p) : W((int64_t)p.tiles * p.kbs), parts(p.ctas) {}
    __device__ __forceinline__ int64_t start(int c) const { return c >= parts ? W : quot(W * c, parts); }
    // the run that holds unit u
    __device__ __forceinline__ int owner(int64_t u) const { return (int)quot((u + 1) * parts - 1, W); }
    // quotient of non-negative numbers, in 32 bits where they fit (a 64-bit division
    // costs some 0.3 us here)
    static __device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
        if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
        return a / b;
    }
};

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

// Epilogue of one product (warps 4-11): the CTA's segments, then the joins of its cut
// tiles. MATS accumulators per segment: 2 (gate, up) or 1. seg: segments so far
// in the launch. False when a wait gave up.
//
// A part is [matrix][T / 4][128 columns] vectors of four tokens, so that a lane
// writes and reads 16 bytes at a time.
// joined() is called once the CTA's outputs are stored, before the tickets are
// released.
template <int MATS, int NT, typename Joined>
__device__ __forceinline__ bool epilogue(const SmallArgs &args, const Product &p, uint32_t *ticket,
                                         SmallCtl *ctl, uint32_t tmem_base, int &seg, Joined joined) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, T = args.T;
    const int set = (warp - 4) >> 2;
    const Runs run(p);
    const int64_t begin = run.start(blockIdx.x), end = run.start(blockIdx.x + 1);
    if (begin == end) return true;
    const bool f16 = args.f16 != 0;
    uint16_t *out = static_cast<uint16_t *>(p.out);
    const int TG = (T + 3) / 4;
    const int64_t part_ld = (int64_t)MATS * TG * 128;  // vectors of one part
    const int first_tile = (int)(begin / p.kbs), last_tile = (int)((end - 1) / p.kbs);
    auto emit = [&](int tile, int t, float s0, float s1) {
        const int col = tile * 128 + q * 32 + lane;
        const float v = MATS == 2 ? s0 * act_sigmoid(s0, args.act) * s1 : s0;
        if (col < p.cols) out[(int64_t)t * p.cols + col] = round16(v, f16);
    };
    auto is_cut = [&](int tile) {
        return begin > (int64_t)tile * p.kbs || end < (int64_t)(tile + 1) * p.kbs;
    };
    // a run's first tile goes to slot 0 of its CTA, a later one (its last) to slot 1
    auto slot = [&](int c, int which) {
        return reinterpret_cast<float4 *>(args.part) + ((int64_t)c * 2 + which) * part_ld + q * 32 + lane;
    };
    // the two tiles that may be cut: the runs [c0, c0 + P) that hold their units, the
    // vectors lo, lo + kSets, .. < hi of tokens that this warp joins, and where c0's part
    // lies
    struct Cut {
        int tile, c0, P, lo, hi;
        const float4 *first;
    } cuts[2];
    int ncuts = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tile = i == 0 ? first_tile : last_tile;
        Cut &x = cuts[i];
        x.tile = -1;
        if ((i == 1 && tile == first_tile) || !is_cut(tile)) continue;
        const int64_t t0 = (int64_t)tile * p.kbs;
        x.tile = tile;
        x.c0 = run.owner(t0);
        x.P = run.owner(t0 + p.kbs - 1) - x.c0 + 1;
        const int k = blockIdx.x - x.c0;
        // (the second tile's vectors go round the sets from the other end)
        x.lo = TG * k / x.P + (i == 0 ? set : kSets - 1 - set);
        x.hi = TG * (k + 1) / x.P;
        x.first = slot(x.c0, run.start(x.c0) == t0 ? 0 : 1);
        ++ncuts;
    }

    for (int tile = first_tile; tile <= last_tile; ++tile, ++seg) {
        const bool cut = is_cut(tile);
        const int a = seg & 1;
        if (!bounded_wait(ptx::smem_addr(&ctl->tfull[a]), (seg >> 1) & 1, args.err)) return false;
        ptx::tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * 2 * NT;
        float4 *mine = cut ? slot(blockIdx.x, tile == first_tile ? 0 : 1) : nullptr;
#pragma unroll 1
        for (int c = 16 * set; c < NT && c < T; c += 16 * kSets) {
            uint32_t r[MATS][16];
#pragma unroll
            for (int m = 0; m < MATS; ++m) tmem_ld16(taddr + m * NT + c, r[m]);
            if (!cut) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < T)
                        emit(tile, c + j, __uint_as_float(r[0][j]), __uint_as_float(r[MATS - 1][j]));
                continue;
            }
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    if (c + j < T)
                        __stcg(mine + (int64_t)(m * TG + (c + j) / 4) * 128,
                               make_float4(__uint_as_float(r[m][j]), __uint_as_float(r[m][j + 1]),
                                           __uint_as_float(r[m][j + 2]), __uint_as_float(r[m][j + 3])));
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->tempty[a]));
        if (cut) {
            // low half: warps whose parts are written; high half: that need them no more
            const Cut &x = tile == first_tile ? cuts[0] : cuts[1];
            __threadfence();
            __syncwarp();
            // (a warp with no share of the tokens needs none of them)
            if (lane == 0) atomicAdd(ticket + tile * 4 + q, x.hi > x.lo ? 1u : 0x10001u);
        }
    }
    if (ncuts == 0) return true;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Cut &x = cuts[i];
        if (x.tile < 0 || x.lo >= x.hi) continue;
        bool ok = true;
        if (lane == 0)
            ok = word_wait(ticket + x.tile * 4 + q, 0xffffu, (uint32_t)(x.P * kSets), args.err);
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    }
    __syncwarp();  // lane 0's acquires come before every lane's loads (a shuffle orders none)
    constexpr int kBatch = MATS == 2 ? 10 : 16;  // parts in flight
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const Cut x = i == 0 ? cuts[0] : cuts[1];
        if (x.tile < 0) continue;
#pragma unroll 1
        for (int g = x.lo; g < x.hi; g += kSets) {
            float sum[MATS][4] = {};
#pragma unroll 1
            for (int c = 0; c < x.P; c += kBatch) {
                float4 v[MATS][kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int m = 0; m < MATS; ++m)
                        v[m][j] = c + j < x.P ? __ldcg((c + j == 0 ? x.first : slot(x.c0 + c + j, 0)) +
                                                       (int64_t)(m * TG + g) * 128)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int m = 0; m < MATS; ++m) {
                        sum[m][0] += v[m][j].x;
                        sum[m][1] += v[m][j].y;
                        sum[m][2] += v[m][j].z;
                        sum[m][3] += v[m][j].w;
                    }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * g + j < T) emit(x.tile, 4 * g + j, sum[0][j], sum[MATS - 1][j]);
        }
    }
    __syncwarp();  // every lane has its parts
    // this warp's shares are done; the last one of a tile returns its ticket to zero
    auto release = [&](const Cut &x) {
        if (x.tile < 0 || x.lo >= x.hi) return;
        uint32_t *w = ticket + x.tile * 4 + q;
        if (atomicAdd(w, 0x10000u) >> 16 == (uint32_t)(x.P * kSets - 1)) *w = 0;
    };
    joined();
    if (lane == 0) {
        release(cuts[0]);
        release(cuts[1]);
    }
    return true;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
stream_ffn_kernel(const __grid_constant__ SmallMaps maps, const __grid_constant__ SmallArgs args) {
    using G = Geo<NT>;
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
            ptx::mbar_init(ptx::smem_addr(&ctl->tempty[a]), 4 * kSets);
        }
        ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
        ptx::fence_barrier_init();
    }
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), G::kTmem);
        ptx::tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------ producer --
        uint32_t it = 0;
        bool ok = true;
#pragma unroll
        for (int ph = 0; ph < 2; ++ph) {
            const Product &p = args.p[ph];
            const Runs run(p);
            const int64_t begin = run.start(blockIdx.x);
            const int count = (int)(run.start(blockIdx.x + 1) - begin);
            int tile = (int)(begin / p.kbs), kb = (int)(begin - (int64_t)tile * p.kbs);
            auto load_w = [&](uint32_t s, int tl, int k) {
                const uint32_t full = ptx::smem_addr(&ctl->full[s]), dst = base + s * G::kStageBytes;
                ptx::mbar_arrive_expect_tx(full, kWBytes + (ph + 1) * G::kTok);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const CUtensorMap *w = &maps.w[ph == 0 ? m : 2];
                    const int y = ph == 0 ? k * BK : (2 * k + m) * BK;
                    ptx::tma_load_2d(dst + m * kMat, w, full, tl * 128, y);
                    ptx::tma_load_2d(dst + m * kMat + kBox, w, full, tl * 128 + 64, y);
                }
            };
            auto load_x = [&](uint32_t s, int k) {
                const uint32_t full = ptx::smem_addr(&ctl->full[s]);
                const uint32_t dst = base + s * G::kStageBytes + kWBytes;
                if (ph == 0) {
                    ptx::tma_load_2d(dst, &maps.x, full, k * BK, 0);
                } else {
                    ptx::tma_load_2d(dst, &maps.h, full, 2 * k * BK, 0);
                    ptx::tma_load_2d(dst + G::kTok, &maps.h, full, (2 * k + 1) * BK, 0);
                }
            };
            auto next = [&](int &tl, int &k) {
                if (++k == p.kbs) {
                    k = 0;
                    ++tl;
                }
            };
            auto wait_empty = [&](uint32_t i) {
                return bounded_wait(ptx::smem_addr(&ctl->empty[i % S]), ((i / S) & 1u) ^ 1u, args.err);
            };
            int done = 0;
            if (ph == 1 && ok && count > 0) {
                // a ring full of weights, then (once H is complete) its rows
                const int ahead = min(count, S);
                const uint32_t it0 = it;
                const int kb0 = kb;
                for (int j = 0; j < ahead && ok; ++j) {
                    ok = wait_empty(it0 + j);
                    if (!ok) break;
                    load_w((it0 + j) % S, tile, kb);
                    next(tile, kb);
                    ++it;
                }
                // Once most CTAs have their part of H, HBM is nearly idle until the last one
                // has: it fetches the units behind the rings into L2 (earlier, the
                // CTAs still in the first product lose what that takes).
                ok = ok && word_wait_least(args.err + kWordGrid, gridDim.x * kAheadNum / 8, args.err);
                int ptl = tile, pk = kb;
                for (int j = ahead; j < min(count, ahead + kAheadUnits) && ok; ++j) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int x = ptl * 128; x < ptl * 128 + 128; x += 64)
                            if (x < p.cols && (2 * pk + m) * BK < p.K)
                                ptx::tma_prefetch_2d(&maps.w[2], x, (2 * pk + m) * BK);
                    next(ptl, pk);
                }
                ok = ok && word_wait(args.err + kWordGrid, 0xffffffffu, gridDim.x, args.err);
                ptx::fence_proxy_async_global();
                // (after a wait that gave up too: every announced byte arrives)
                int tl = 0, k = kb0;
                for (uint32_t i = it0; i < it; ++i) {
                    load_x(i % S, k);
                    next(tl, k);
                }
                done = ahead;
            }
            for (int j = done; j < count && ok; ++j) {
                ok = wait_empty(it);
                if (!ok) break;
                load_w(it % S, tile, kb);
                load_x(it % S, kb);
                next(tile, kb);
                ++it;
            }
        }
        if (!ok) {
            // drain the loads that may still be landing in shared memory
            const uint32_t first = it > (uint32_t)S ? it - S : 0u;
            for (uint32_t j = first; j < it; ++j)
                bounded_wait(ptx::smem_addr(&ctl->full[j % S]), (j / S) & 1u, args.err);
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------------------------------------------- MMA issuer --
        uint32_t it = 0;
        int seg = 0;
        bool ok = true;
#pragma unroll
        for (int ph = 0; ph < 2; ++ph) {
            const Product &p = args.p[ph];
            const Runs run(p);
            const int64_t begin = run.start(blockIdx.x);
            const int count = (int)(run.start(blockIdx.x + 1) - begin);
            int kb = (int)(begin % p.kbs);
            bool first = true;
            for (int j = 0; j < count && ok; ++j, ++it) {
                const uint32_t s = it % S, a = seg & 1;
                if (first) {
                    ok = bounded_wait(ptx::smem_addr(&ctl->tempty[a]), ((seg >> 1) & 1) ^ 1, args.err);
                    if (!ok) break;
                    ptx::tc_fence_after();
                }
                ok = bounded_wait(ptx::smem_addr(&ctl->full[s]), (it / S) & 1u, args.err);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t sW = base + s * G::kStageBytes, sX = sW + kWBytes;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        // gate/up: two matrices, two accumulators, the same tokens; down:
                        // two successive halves of the reduction, one accumulator
                        const uint64_t bd =
                            ptx::desc_sw128(sX + (ph == 0 ? 0 : m * G::kTok) + k * 32, 16, 1024);
                        ptx::tc_mma_f16(tmem_base + a * 2 * NT + (ph == 0 ? m * NT : 0),
                                        ptx::desc_sw128(sW + m * kMat + k * 2048, kBox, 1024), bd,
                                        args.idesc, !first || k != 0 || (ph == 1 && m != 0));
                    }
                ptx::tc_commit(ptx::smem_addr(&ctl->empty[s]));
                first = false;
                if (++kb == p.kbs || j == count - 1) {
                    ptx::tc_commit(ptx::smem_addr(&ctl->tfull[a]));
                    ++seg;
                    kb = 0;
                    first = true;
                }
            }
        }
        ptx::tc_commit(ptx::smem_addr(&ctl->drain));
        bounded_wait(ptx::smem_addr(&ctl->drain), 0, args.err);
    } else if (warp >= 4) {
        // ------------------------------------------------------ epilogue --
        int seg = 0;
        bool arrived = false;
        auto arrive = [&] {
            if (arrived) return;
            arrived = true;
            // this CTA's part of H is complete and visible to the loads of all SMs
            ptx::fence_proxy_async_global();
            __threadfence();
            asm volatile("bar.sync 1, %0;" ::"n"(128 * kSets) : "memory");
            if (warp == 4 && lane == 0) atomicAdd(args.err + kWordGrid, 1u);
        };
        const bool ok = epilogue<2, NT>(args, args.p[0], args.ticket, ctl, tmem_base, seg, arrive);
        arrive();  // (without a cut tile, or after a wait that gave up)
        if (ok)
            epilogue<1, NT>(args, args.p[1], args.ticket + 4 * args.p[0].tiles, ctl, tmem_base, seg,
                            [] {});
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc(tmem_base, G::kTmem);
    if (tid == 0) {
        // the last CTA to leave returns the grid's counters to zero
        __threadfence();
        if (atomicAdd(args.err + kWordExit, 1u) == gridDim.x - 1) {
            args.err[kWordGrid] = 0;
            args.err[kWordExit] = 0;
        }
    }
}

template <int NT>
cudaError_t launch_nt(const SmallMaps &maps, SmallArgs args, int grid, cudaStream_t s) {
    constexpr size_t kSmem = Geo<NT>::kSmem;
    args.idesc = idesc(args.f16 != 0, 128, NT, true, false);
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(stream_ffn_kernel<NT>), (int)kSmem);
    if (e != cudaSuccess) return e;
    return launch_together(stream_ffn_kernel<NT>, dim3(grid), dim3(kThreads), kSmem, s, maps, args);
}

int padded_tokens(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

// A product whose units are 32 KB of weights, on one CTA per SM, fewer where a run
// would be under two units (then the joining costs more than the shorter runs save).
Product make_product(int cols, int K, int depth, int sms, void *out) {
    Product p;
    p.cols = cols;
    p.K = K;
    p.kbs = (K + depth - 1) / depth;
    p.tiles = (cols + 127) / 128;
    p.ctas = (int)std::min<int64_t>(std::min(sms, kFfnMaxCtas),
                                    std::max<int64_t>(p.tiles, (int64_t)p.tiles * p.kbs / 2));
    p.out = out;
    return p;
}

}  // namespace
}  // namespace ffn

using namespace ffn;

size_t ffn_stream_part_bytes(int T, int d, int n) {
    // two parts for each CTA, of two matrices in the first product
    const size_t ctas = std::max(2 * make_product(n, d, BK, kFfnMaxCtas, nullptr).ctas,
                                 make_product(d, n, 2 * BK, kFfnMaxCtas, nullptr).ctas);
    return ctas * 2 * ((T + 3) / 4) * 128 * 4 * sizeof(float);
}

cudaError_t launch_ffn_stream(const void *X, const void *W1, const void *W3, const void *W2, int T,
                              int d, int n, int act, bool f16, void *H, void *Y, float *part,
                              uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    const int nt = padded_tokens(T);
    SmallMaps m{};
    const CUtensorMapDataType ty = map_type(f16);
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    if (!make_map(&m.w[0], ty, W1, n, d, 64, BK, sw) || !make_map(&m.w[1], ty, W3, n, d, 64, BK, sw) ||
        !make_map(&m.w[2], ty, W2, d, n, 64, BK, sw) || !make_map(&m.x, ty, X, d, T, 64, nt, sw) ||
        !make_map(&m.h, ty, H, n, T, 64, nt, sw))
        return cudaErrorInvalidValue;
    SmallArgs a{};
    a.p[0] = make_product(n, d, BK, sm_count(), H);
    a.p[1] = make_product(d, n, 2 * BK, sm_count(), Y);
    a.T = T;
    a.act = act;
    a.f16 = f16;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    const int grid = std::max(a.p[0].ctas, a.p[1].ctas);
    switch (nt) {
        case 16: return launch_nt<16>(m, a, grid, s);
        case 32: return launch_nt<32>(m, a, grid, s);
        default: return launch_nt<64>(m, a, grid, s);
    }
}

}  // namespace moe
