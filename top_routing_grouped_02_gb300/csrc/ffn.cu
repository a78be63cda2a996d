// Dense gated feed-forward block on the 5th-generation tensor cores, forward and
// backward:
//   A1 = X W1, A3 = X W3, H = act(A1) * A3, Y = H W2
//   G = dY W2^T, dA1 = G F1, dA3 = G F3, where F1 = A3 act'(A1), F3 = act(A1)
//   dX = dA1 W1^T + dA3 W3^T, dW1 = X^T dA1, dW3 = X^T dA3, dW2 = H^T dY
// X, Y [T,d], W1, W3 [d,n], W2 [n,d], all 16 bits; accumulation in fp32.
//
// One persistent kernel template runs all five products (Mode). Each is bound by
// the tensor cores once T is a few hundred; few tokens take the weight-streaming
// kernel of ffn_small.cu instead. A CTA pair (tcgen05 cta_group::2) owns a tile
// of 256 rows x 256 columns: each CTA holds its 128 rows of A and half of the
// columns of B per 64-deep stage, the even CTA issues the MMAs over both. Two
// accumulators in TMEM: the epilogue of one tile runs while the MMAs fill the
// other. gate/up: the even CTA's half of B is W1's columns and the odd CTA's W3's,
// so a thread finds a1 and a3 of one element in its own TMEM lane and H leaves in
// the epilogue; neither A1 nor A3 is read back from memory in the forward.
// Tiles rarely come out even over the SM pairs. Where the tiles past the last whole wave
// (or all, if they are few) leave half of the pairs idle or more, each is cut along the
// reduction into as many equal segments as there are pairs for it (split_work). The
// pairs that hold a tile's segments join them: every epilogue warp writes its sums
// (fp32) to the workspace, but for its own share of the columns, and once all have, each
// adds its share, in the order of the segments: the result does not depend on timing.
// The cut tiles come first in each pair's work, so that joining overlaps whole tiles.
// (Equal runs over all of the last tiles, cut anywhere, balance better and measured
// slower: pairs that share operands then read them at different places of the
// reduction, 746 against 571 us for dX of 4096 tokens, d = 4096, n = 14336.)
// Measured, 4096 tokens, d = 4096, n = 14336 bf16 under the power cap: gate/up 570-600 us
// (1.6-1.7 PFLOP/s), down 270-280, dA1 and dA3 300-310, dX 530-550, weight gradients
// 770-800. 777 tokens, 1000 x 2728: 24.5, 15, 16.5, 19 and 19.5 us, of which a pair's longest
// run of k-blocks (32, 11, 16, 22 and 26, at 0.33 us each; gate and the weight gradients are
// two waves) takes 10.7, 3.7, 5.3, 7.3 and 8.7; the rest is the start (1 us), the ring's fill
// (2-3), the last epilogue (1.5-4) or the join (5), and the end (1.5).
// The projections (kLinear and the products of its gradients): 4096 tokens, 4096 x 14336 bf16 with
// F 285 us (1.69 PFLOP/s), dX 256 (1.88), dW 248 (1.94); 777 tokens, 1000 x 2728: 19 us with F, bias,
// gelu and residual (12.4 with none of them), dX and dW together 20; 512 tokens, 7168 x 2048 fp16:
// 24 us.
// All tails (T, d, n need not be multiples of a tile) are left to TMA: loads
// outside a tensor give zeros, which add nothing, and stores outside write nothing.
//
// The backward's operands dA1, dA3 and the forward's H are rounded to 16 bits
// because the tensor cores multiply 16-bit operands. The factors F1 and F3 are made by
// the forward, where the sigmoid is at hand, and kept in fp32 (in blocks, see
// saved_block), so that dA1 and dA3 carry one rounding each and not three.
//
// Warps: 0 TMA producer, 1 MMA issuer (even CTA), 2 TMEM allocation, 4-11 epilogue
// (two warps per quadrant of 32 TMEM lanes, splitting the columns). Waits are
// bounded; a wait that gives up flags the error word, its role stops, and loads and
// MMAs in flight are drained before the CTA leaves.
#include <algorithm>
#include <type_traits>

#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols,
              uint64_t rows, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return nullptr;
    }();
    if (fn == nullptr) return false;
    const uint64_t es = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * es};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// kGate: H (and, for training, F1, F3) from X, W1, W3. kDown: Y from H, W2.
// kDHid: dA1, dA3 from dY, W2 (K-major: its rows are the output columns) and F1,
// F3. kDX: dX, one reduction over dA1 W1^T then dA3 W3^T (K-major weights).
// kWGrad: dW1, dW3, dW2 in one launch, both operands MN-major, reduction over T.
// kLinear: a projection, Y = act(X W + bias) + residual, and (training) F = act'(X W + bias);
// its gradients are products of the modes kDX, with no second half, and kWGrad, with one problem,
// or both in one launch (kBoth: problem 0 is dX, problem 1 is dW) where both are small.
enum Mode : int { kGate = 0, kDown = 1, kDHid = 2, kDX = 3, kWGrad = 4, kLinear = 5, kBoth = 6 };

constexpr int BM = 128;  // rows per CTA
constexpr int BK = 64;   // reduction depth per stage: 128 bytes of 16-bit elements
constexpr int kEpiWarps = 8;
constexpr int kShares = kEpiWarps / 4;  // warps of one quadrant share the columns
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kABytes = BM * BK * 2;  // 16 KB
constexpr uint32_t kBox = 64 * 64 * 2;     // 8 KB: 64 x 64 elements
constexpr uint32_t kEpiBuf = 32 * 64;      // 32 rows of 64 bytes
constexpr int kEpiBufs = 2;                // per epilogue warp
// Row-tile pairs that take every column block before the next group starts: the
// 76 pairs at work then cover about 8 x 10 tiles and share their operands in L2.
constexpr int kGroup = 8;

constexpr int BN = 256;                      // tile columns
constexpr int kBoxes = BN / 128;             // 64-column boxes of B per CTA
constexpr uint32_t kStageBytes = kABytes + kBoxes * kBox;
constexpr int kStages = 6;                   // 192 KB
constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes +
                         (size_t)kEpiWarps * kEpiBufs * kEpiBuf + 256;
// Vectors (float4) of one warp's part: its columns of 32 rows.
constexpr int kPartVecs = BN / kShares * 32 / 4;

// Up to this many segments a cut tile is joined in boxes of 32 columns, which leave by
// TMA; more, four columns at a time, so that all holders have a share and eight segments
// are in flight (24 segments, 66 tokens: 20.4 -> 14.8 us; three, 3133 tokens: 19.7 -> 25.4).
constexpr int kFewSegments = 4;

struct Maps {
    CUtensorMap a[3], b[3], o[3];
};

struct Args {
    int units;           // tiles of all problems
    int cut, split;      // the first `cut` of them are cut into `split` segments each
    int first[3];        // first unit of each problem (kWGrad: three, else one)
    int mt[3], nb[3];    // row-tile pairs, column blocks
    int rows[3], cols[3];// of the outputs
    int kb, kb_half;     // k-blocks; kDX: those of its first half
    int kb_dw;           // kBoth: those of problem 1
    uint32_t idesc, idesc_dw;
    int f16, act;
    void *out[3];        // the outputs of each problem (kDHid: both of its one)
    const void *bias;    // kLinear: [cols] of 16 bits or (bias32) fp32, or NULL
    int bias32;
    const void *res;     // kLinear: [rows, cols] of 16 bits, or NULL; out[0] may be it
    // kWGrad and kBoth of a projection: its bias' gradient [sum_n] (of 16 bits or (bias32) fp32, or NULL),
    // the sums of sum_rows rows of sums [.][sum_n]
    void *dbias;
    const float *sums;
    int sum_rows, sum_n;
    float *f1, *f3;      // the factors in blocks (saved_block): kGate stores them, or
                         // NULL; kDHid reads them; kLinear stores F in f1, or NULL
    float4 *part;        // [segment][CTA][warp][kPartVecs]
    uint32_t *ticket;    // [cut][CTA][warp]
    uint32_t *err;
};

// The factors F1, F3 [T, n] fp32 in blocks of 32 x 32: lane r of an epilogue
// warp holds row r of a block, so that a block is 8 x 32 vectors of four columns, and
// a warp stores and loads 512 consecutive bytes an instruction. (As rows, each
// instruction touches 32 lines, and the 16 loads of a block took as long as the main
// loop of a short reduction.)
__device__ __forceinline__ float4 *saved_block(float *a, int n, int row, int col, int lane) {
    const int64_t block = (int64_t)(row / 32) * ((n + 31) / 32) + col / 32;
    return reinterpret_cast<float4 *>(a) + block * 256 + lane;
}

// Two neighbouring words as a pair of fp32 values, and back.
__device__ __forceinline__ f32x2 word_pair(const uint32_t *w) {
    return pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
}
__device__ __forceinline__ void put_pair(f32x2 p, uint32_t *w) {
    float x, y;
    unpair(p, x, y);
    w[0] = __float_as_uint(x);
    w[1] = __float_as_uint(y);
}

__device__ __forceinline__ f32x2 pair2(const float *f) { return pair(f[0], f[1]); }
__device__ __forceinline__ float4 pairs_float4(f32x2 a, f32x2 b) {
    float4 r;
    unpair(a, r.x, r.y);
    unpair(b, r.z, r.w);
    return r;
}
__device__ __forceinline__ float4 words_float4(const uint32_t *w) {
    return make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                       __uint_as_float(w[3]));
}

struct Ctl {
    uint64_t full[8], empty[8], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
};
static_assert(sizeof(Ctl) <= 256, "control block");

// A pair's work: its segment of a cut tile, if it has one (pair = tile * split +
// segment), then whole tiles.
struct Work {
    int pairs, units, kb, next;
    int dw, kb_dw;    // kBoth: problem 1's first tile, its k-blocks
    int u, kb0, kb1;  // current: tile, its k-blocks
    bool cut;         // a segment
    __device__ __forceinline__ Work(const Args &a, int pair, int pairs_)
        : pairs(pairs_), units(a.units), kb(a.kb), next(a.cut + pair), dw(a.first[1]), kb_dw(a.kb_dw), cut(false) {
        if (pair < a.cut * a.split) {
            u = pair / a.split;
            const int j = pair - u * a.split;
            kb0 = (int)((int64_t)kb * j / a.split);
            kb1 = (int)((int64_t)kb * (j + 1) / a.split);
            cut = true;
        }
    }
    bool started = false;
    __device__ __forceinline__ bool step() {
        if (cut && !started) return started = true;
        cut = false;
        if (next >= units) return false;
        u = next;
        next += pairs;
        kb0 = 0;
        kb1 = kb_dw > 0 && u >= dw ? kb_dw : kb;
        return true;
    }
};

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
dense_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args args) {
    constexpr int S = kStages;
    // whether A's tiles have the rows as the contiguous dimension, and B's the reduction
    auto a_mn = [](int p) { return MODE == kWGrad || (MODE == kBoth && p == 1); };
    auto b_k = [](int p) { return MODE == kDHid || MODE == kDX || (MODE == kBoth && p == 0); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + (size_t)S * kStageBytes +
                                       (size_t)kEpiWarps * kEpiBufs * kEpiBuf);
    const uint32_t base = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&ctl->tfull[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctl->tempty[a]), 2 * kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
        ptx::fence_barrier_init();
    }
    if (warp == 3 && lane < 9) {  // the descriptors of this mode's tensors
        constexpr int nA = MODE == kWGrad ? 3 : MODE == kDX || MODE == kBoth ? 2 : 1;
        constexpr int nB = MODE == kWGrad ? 3 : MODE == kDX || MODE == kGate || MODE == kBoth ? 2 : 1;
        constexpr int nO = MODE == kWGrad ? 3 : MODE == kDHid || MODE == kBoth ? 2 : 1;
        const int k = lane % 3;
        if (lane < 3 ? k < nA : lane < 6 ? k < nB : k < nO)
            ptx::prefetch_tensormap(lane < 3 ? &maps.a[k] : lane < 6 ? &maps.b[k] : &maps.o[k]);
    }
    if (warp == 2) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base), 2 * BN);
        ptx::tmem_relinquish_pair();
    }
    pdl_wait();
    pdl_trigger();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;

    struct Unit {
        int p, m, nb, row0;  // problem, row-tile pair, column block, this CTA's first row
    };
    auto unit_at = [&](int u) {
        Unit x;
        x.p = 0;
        if (MODE == kWGrad) x.p = u >= args.first[2] ? 2 : u >= args.first[1] ? 1 : 0;
        if (MODE == kBoth) x.p = u >= args.first[1] ? 1 : 0;
        u -= args.first[x.p];
        const int mt = args.mt[x.p], per = kGroup * args.nb[x.p];
        const int k = u / per, gs = min(kGroup, mt - k * kGroup), r = u - k * per;
        x.nb = r / gs;
        x.m = k * kGroup + r - x.nb * gs;
        x.row0 = (2 * x.m + (int)rank) * BM;
        return x;
    };

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------ producer --
        uint32_t it = 0;
        bool ok = true;
        for (Work w(args, pair, pairs); ok && w.step();) {
            const Unit un = unit_at(w.u);
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const uint32_t s = it % S;
                if (!bounded_wait(ptx::smem_addr(&ctl->empty[s]), ((it / S) & 1u) ^ 1u, args.err)) {
                    ok = false;
                    break;
                }
                // both CTAs' loads complete on the even CTA's barrier
                const uint32_t full = ptx::smem_addr(&ctl->full[s]);
                if (leader) ptx::mbar_arrive_expect_tx(full, 2 * kStageBytes);
                const uint32_t bar = ptx::mapa(full, 0);
                const uint32_t sA = base + s * kStageBytes, sB = sA + kABytes;
                const bool second = MODE == kDX && kb >= args.kb_half;
                const int k0 = (second ? kb - args.kb_half : kb) * BK;
                const int ai = MODE == kWGrad || MODE == kBoth ? un.p : second ? 1 : 0;
                const int bi = MODE == kWGrad || MODE == kBoth ? un.p
                               : MODE == kGate ? (int)rank
                               : second ? 1 : 0;
                if (a_mn(un.p)) {
                    ptx::tma_load_2d_pair(sA, &maps.a[ai], bar, un.row0, k0);
                    ptx::tma_load_2d_pair(sA + kBox, &maps.a[ai], bar, un.row0 + 64, k0);
                } else {
                    ptx::tma_load_2d_pair(sA, &maps.a[ai], bar, k0, un.row0);
                }
                // this CTA's half of the tile's columns of B
                const int c0 = MODE == kGate ? un.nb * (BN / 2) : un.nb * BN + (int)rank * (BN / 2);
#pragma unroll
                for (int q = 0; q < kBoxes; ++q) {
                    if (b_k(un.p)) ptx::tma_load_2d_pair(sB + q * kBox, &maps.b[bi], bar, k0, c0 + q * 64);
                    else ptx::tma_load_2d_pair(sB + q * kBox, &maps.b[bi], bar, c0 + q * 64, k0);
                }
            }
        }
        if (!ok && leader) {
            const uint32_t first = it > (uint32_t)S ? it - S : 0u;
            for (uint32_t j = first; j < it; ++j)
                bounded_wait(ptx::smem_addr(&ctl->full[j % S]), (j / S) & 1u, args.err);
        }
    } else if (warp == 1 && lane == 0 && leader) {
        // ---------------------------------------------------- MMA issuer --
        uint32_t it = 0, uc = 0;
        bool ok = true;
        for (Work w(args, pair, pairs); ok && w.step(); ++uc) {
            const uint32_t a = uc & 1u;
            const int prob = MODE == kBoth && w.u >= args.first[1] ? 1 : 0;
            const uint32_t idesc = prob == 1 ? args.idesc_dw : args.idesc;
            if (!bounded_wait(ptx::smem_addr(&ctl->tempty[a]), ((uc >> 1) & 1u) ^ 1u, args.err)) break;
            ptx::tc_fence_after();
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const uint32_t s = it % S;
                if (!bounded_wait(ptx::smem_addr(&ctl->full[s]), (it / S) & 1u, args.err)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t sA = base + s * kStageBytes, sB = sA + kABytes;
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                    // K-major: the next 16 of the reduction are 32 bytes on; MN-major:
                    // 16 rows of 128 bytes, 64-column slabs 8 KB apart
                    const uint64_t ad = a_mn(prob) ? ptx::desc_sw128(sA + k * 2048, kBox, 1024)
                                             : ptx::desc_sw128(sA + k * 32, 16, 1024);
                    const uint64_t bd = b_k(prob) ? ptx::desc_sw128(sB + k * 32, 16, 1024)
                                            : ptx::desc_sw128(sB + k * 2048, kBox, 1024);
                    ptx::tc_mma_f16_pair(tmem_base + a * BN, ad, bd, idesc, kb != w.kb0 || k != 0);
                }
                ptx::tc_commit_pair(ptx::smem_addr(&ctl->empty[s]), 0x3);
            }
            if (!ok) break;
            ptx::tc_commit_pair(ptx::smem_addr(&ctl->tfull[a]), 0x3);
        }
        ptx::tc_commit_pair(ptx::smem_addr(&ctl->drain), 0x1);
        bounded_wait(ptx::smem_addr(&ctl->drain), 0, args.err);
    } else if ((MODE == kWGrad || MODE == kBoth) && warp == 3) {
        // the bias' gradient beside the products: a launch of its own took 2 us of a short
        // training step's 55
        if (args.dbias != nullptr)
            for (int c = blockIdx.x * 32 + lane; c < args.sum_n; c += gridDim.x * 32) {
                float v = 0.f;
#pragma unroll 8
                for (int p = 0; p < args.sum_rows; ++p) v += __ldg(args.sums + (int64_t)p * args.sum_n + c);
                if (args.bias32) static_cast<float *>(args.dbias)[c] = v;
                else static_cast<uint16_t *>(args.dbias)[c] = round16(v, args.f16 != 0);
            }
    } else if (warp >= 4) {
        // ------------------------------------------------------ epilogue --
        const int ew = warp - 4, q = warp & 3, share = ew >> 2;
        const uint32_t buf0 = base + (uint32_t)S * kStageBytes + (uint32_t)ew * kEpiBufs * kEpiBuf;
        const uint32_t tempty0 = ptx::mapa(ptx::smem_addr(&ctl->tempty[0]), 0);
        const bool f16 = args.f16 != 0;
        uint32_t groups = 0, uc = 0;
        // 32 rows x 64 bytes through a staging buffer (64-byte swizzle) and a TMA store at
        // (x, y)
        auto store_box = [&](const uint32_t (&v)[16], int x, int y, const CUtensorMap *map) {
            const uint32_t buf = buf0 + (groups % kEpiBufs) * kEpiBuf;
            if (lane == 0 && groups >= (uint32_t)kEpiBufs) ptx::bulk_wait_group_read<kEpiBufs - 1>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ptx::st_shared_v4(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), v[4 * i],
                                  v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(map, buf, x, y);
                ptx::bulk_commit_group();
            }
            ++groups;
        };
        constexpr int kCols = MODE == kGate ? BN / 2 : BN;  // output columns of a tile
        constexpr int NC = kCols / kShares / 32;            // 32-column chunks of a warp
        const int c_lo = share * NC;
        // A cut tile. A warp's part is kPartVecs / 32 vectors of four columns x 32 rows; a
        // unit of the join is such a vector (kGate: of W1's sums and of W3's). Each warp
        // writes its part, but for the units that it joins itself: its pair's share, which
        // goes round the warps where there are more segments than units.
        constexpr int M = MODE == kGate ? 2 : 1, NU = kPartVecs / 32 / M;
        auto part_of = [&](int p) {
            return args.part + (((int64_t)p * 2 + rank) * kEpiWarps + ew) * kPartVecs + lane;
        };
        // the accumulator's column of vector v of this warp's part
        auto column = [&](int v) {
            return MODE == kGate ? (v / NU) * (BN / 2) + share * NU * 4 + v % NU * 4 : share * NU * 4 + v * 4;
        };
        // kLinear: the bias of four columns; a call with the activation and whether its
        // derivative is wanted, known at compile time
        auto bias_pairs = [&](int x, f32x2 (&b)[2]) {
            if (args.bias32) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(args.bias) + x));
                b[0] = moe::pair(q.x, q.y);
                b[1] = moe::pair(q.z, q.w);
                return;
            }
            const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(args.bias) + x));
            float f[4];
            if (f16) {
                unpack2<__half>(q.x, f[0], f[1]);
                unpack2<__half>(q.y, f[2], f[3]);
            } else {
                unpack2<__nv_bfloat16>(q.x, f[0], f[1]);
                unpack2<__nv_bfloat16>(q.y, f[2], f[3]);
            }
            b[0] = pair2(f);
            b[1] = pair2(f + 2);
        };
        auto with_act = [&](auto &&call) {
            using yes = std::true_type;
            using no = std::false_type;
            if (args.act == kNoAct) call(std::integral_constant<int, kNoAct>(), no());
            else if (args.act == MOE_ACT_SILU)
                args.f1 != nullptr ? call(std::integral_constant<int, MOE_ACT_SILU>(), yes())
                                   : call(std::integral_constant<int, MOE_ACT_SILU>(), no());
            else
                args.f1 != nullptr ? call(std::integral_constant<int, MOE_ACT_GELU_TANH>(), yes())
                                   : call(std::integral_constant<int, MOE_ACT_GELU_TANH>(), no());
        };
        // 32 columns of this pair's cut tile from its segments, in their order, this pair's
        // own from its accumulator (column col); v0: their first vector in the parts
        auto gather = [&](int v0, uint32_t taddr, int col, uint32_t (&v)[32]) {
            float s[32] = {};
            const int p0 = pair - pair % args.split;
#pragma unroll 1
            for (int p = p0; p < p0 + args.split; ++p) {
                if (p == pair) {
                    ptx::tmem_ld32(taddr + col, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] += __uint_as_float(v[i]);
                    continue;
                }
                const float4 *src = part_of(p) + v0 * 32;
                float4 q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = __ldcg(src + i * 32);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[4 * i] += q[i].x;
                    s[4 * i + 1] += q[i].y;
                    s[4 * i + 2] += q[i].z;
                    s[4 * i + 3] += q[i].w;
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(s[i]);
        };
        // The chunks [lo, hi) of this warp's columns of a tile to the outputs: from the
        // accumulator at taddr alone, or joined from the tile's segments. ready(): waits for
        // either; release(): called after the last read of the accumulator.
        auto finish = [&](const Unit &un, int lo, int hi, uint32_t taddr, bool joined, auto ready,
                          auto release) {
            const int rows = args.rows[un.p], cols = args.cols[un.p];
            const int y0 = un.row0 + q * 32;
            // chunks that are not all outside
            hi = y0 < rows ? min(hi, (cols - un.nb * kCols + 31) / 32) : 0;
            // kDHid: this row's factors of a chunk, loaded while the one before is stored
            float4 x1[8] = {}, x3[8] = {};
            auto load_factors = [&](int c) {
                if (c >= hi) return;
                const int x0 = un.nb * kCols + c * 32;
                const float4 *p1 = saved_block(args.f1, cols, y0, x0, lane);
                const float4 *p3 = saved_block(args.f3, cols, y0, x0, lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x1[i] = __ldg(p1 + i * 32);
                    x3[i] = __ldg(p3 + i * 32);
                }
            };
            // kLinear: this row's residual of a chunk, loaded a chunk ahead, and the bias of four of
            // the warp's columns, which a shuffle hands out (777 x 1000 x 2728: loads where they
            // are used cost 1.7 and 3.7 of 18.2 us)
            [[maybe_unused]] uint4 rr[4] = {}, ahead[4] = {};
            [[maybe_unused]] f32x2 bias4[2] = {0, 0};
            auto load_residual = [&](int c, uint4 (&rr)[4]) {
                if (args.res == nullptr || c >= hi || y0 + lane >= rows) return;
                const int x0 = un.nb * kCols + c * 32;
                const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(args.res) +
                                                                 (int64_t)(y0 + lane) * cols + x0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (x0 + 8 * i < cols) rr[i] = p[i];
            };
            if constexpr (MODE == kDHid) load_factors(lo);
            if constexpr (MODE == kLinear) {
                const int x = un.nb * kCols + c_lo * 32 + lane * 4;
                if (args.bias != nullptr && x < cols) bias_pairs(x, bias4);
                load_residual(lo, rr);
            }
            if (!ready()) return false;
            if (lo >= hi) release();
            // m: W1's sums or (kGate) W3's
            auto load = [&](int c, int m, uint32_t (&v)[32]) {
                const int col = m * (BN / 2) + c * 32;
                if (joined) gather(m * NU + (c - c_lo) * 8, taddr, col, v);
                else ptx::tmem_ld32(taddr + col, v);
            };
#pragma unroll 1
            for (int c = lo; c < hi; ++c) {
                const int x0 = un.nb * kCols + c * 32;
                if constexpr (MODE == kGate) {
                    uint32_t g[32], v[32], o[16];
                    load(c, 0, g);
                    load(c, 1, v);
                    if (c == hi - 1) release();
                    const bool train = args.f1 != nullptr;
                    auto chunk = [&](auto gelu, auto saves) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            f32x2 h, f1 = 0, f3;
                            activate<gelu(), saves()>(word_pair(g + 2 * i), word_pair(v + 2 * i), h, f1, f3);
                            float x, y;
                            unpair(h, x, y);
                            o[i] = pack(x, y, f16);
                            if (saves()) {
                                put_pair(f1, v + 2 * i);
                                put_pair(f3, g + 2 * i);
                            }
                        }
                    };
                    using yes = std::true_type;
                    using no = std::false_type;
                    if (args.act == MOE_ACT_SILU) train ? chunk(no(), yes()) : chunk(no(), no());
                    else train ? chunk(yes(), yes()) : chunk(yes(), no());
                    // v: F1, g: F3
                    store_box(o, x0, y0, &maps.o[0]);
                    if (train) {
                        float4 *p1 = saved_block(args.f1, cols, y0, x0, lane);
                        float4 *p3 = saved_block(args.f3, cols, y0, x0, lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            p1[i * 32] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                     __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                            p3[i * 32] = make_float4(__uint_as_float(g[4 * i]), __uint_as_float(g[4 * i + 1]),
                                                     __uint_as_float(g[4 * i + 2]), __uint_as_float(g[4 * i + 3]));
                        }
                    }
                } else if constexpr (MODE == kDHid) {
                    uint32_t g[32], o1[16], o3[16];
                    load(c, 0, g);
                    if (c == hi - 1) release();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float *r1 = &x1[i >> 1].x + 2 * (i & 1), *r3 = &x3[i >> 1].x + 2 * (i & 1);
                        const float g0 = __uint_as_float(g[2 * i]), g1 = __uint_as_float(g[2 * i + 1]);
                        o1[i] = pack(g0 * r1[0], g1 * r1[1], f16);
                        o3[i] = pack(g0 * r3[0], g1 * r3[1], f16);
                    }
                    load_factors(c + 1);
                    store_box(o1, x0, y0, &maps.o[0]);
                    store_box(o3, x0, y0, &maps.o[1]);
                } else if constexpr (MODE == kLinear) {
                    uint32_t v[32], o[16];
                    load_residual(c + 1, ahead);
                    load(c, 0, v);
                    if (c == hi - 1) release();
                    if (args.bias != nullptr) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const f32x2 b = __shfl_sync(0xffffffffu, bias4[i & 1], (c - c_lo) * 8 + (i >> 1));
                            put_pair(add2(word_pair(v + 2 * i), b), v + 2 * i);
                        }
                    }
                    auto chunk = [&](auto act, auto saves) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            f32x2 f, df = 0;
                            activate_one<act(), saves()>(word_pair(v + 2 * i), f, df);
                            float x, y;
                            if (args.res != nullptr) {
                                const uint32_t w = (&rr[i >> 2].x)[i & 3];
                                if (f16) unpack2<__half>(w, x, y);
                                else unpack2<__nv_bfloat16>(w, x, y);
                                f = add2(f, moe::pair(x, y));
                            }
                            unpair(f, x, y);
                            o[i] = pack(x, y, f16);
                            if (saves()) put_pair(df, v + 2 * i);
                        }
                    };
                    with_act(chunk);
#pragma unroll
                    for (int i = 0; i < 4; ++i) rr[i] = ahead[i];
                    store_box(o, x0, y0, &maps.o[0]);
                    if (args.f1 != nullptr) {
                        float4 *p = saved_block(args.f1, cols, y0, x0, lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i) p[i * 32] = words_float4(v + 4 * i);
                    }
                } else {
                    uint32_t v[32], o[16];
                    load(c, 0, v);
                    if (c == hi - 1) release();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), f16);
                    store_box(o, x0, y0, &maps.o[MODE == kWGrad || MODE == kBoth ? un.p : 0]);
                }
            }
            return true;
        };

        // The join of many segments: units [lo, hi), one after the other, each the sum of its
        // segments in their order, eight in flight.
        auto join = [&](const Unit &un, uint32_t taddr, int lo, int hi) {
            constexpr int P = 8;
            const int rows = args.rows[un.p], cols = args.cols[un.p];
            const int y = un.row0 + q * 32, x_lo = un.nb * kCols + share * NU * 4;
            const int p0 = pair - pair % args.split;
            hi = min(hi, (cols - x_lo + 3) / 4);
#pragma unroll 1
            for (int u = lo; u < hi; ++u) {
                const int x = x_lo + u * 4;
                auto saved = [&](float *f) {
                    return saved_block(f, cols, y, x, lane) + (x & 31) / 4 * 32;
                };
                [[maybe_unused]] float4 f1, f3;
                [[maybe_unused]] f32x2 bias[2] = {0, 0};
                [[maybe_unused]] uint2 res = {0, 0};
                if constexpr (MODE == kLinear) {
                    if (args.bias != nullptr) bias_pairs(x, bias);
                    if (args.res != nullptr && y + lane < rows)
                        res = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(args.res) +
                                                               (int64_t)(y + lane) * cols + x);
                }
                if constexpr (MODE == kDHid) {
                    f1 = __ldg(saved(args.f1));
                    f3 = __ldg(saved(args.f3));
                }
                float s[M][4] = {};
#pragma unroll 1
                for (int pb = 0; pb < args.split; pb += P) {
                    float4 v[P][M];
#pragma unroll
                    for (int k = 0; k < P; ++k)
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            v[k][m] = pb + k < args.split && p0 + pb + k != pair
                                          ? __ldcg(part_of(p0 + pb + k) + (m * NU + u) * 32)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                    const int mine = pair - p0 - pb;  // this pair's own comes from the accumulator
                    if (mine >= 0 && mine < P) {
#pragma unroll
                        for (int m = 0; m < M; ++m) {
                            uint32_t r[4];
                            tmem_ld4(taddr + column(m * NU + u), r);
#pragma unroll
                            for (int k = 0; k < P; ++k)
                                if (k == mine) v[k][m] = words_float4(r);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < P; ++k)
#pragma unroll
                        for (int m = 0; m < M; ++m) {
                            s[m][0] += v[k][m].x;
                            s[m][1] += v[k][m].y;
                            s[m][2] += v[k][m].z;
                            s[m][3] += v[k][m].w;
                        }
                }
                if (y + lane < rows) {
                    auto store = [&](int k, f32x2 a, f32x2 b) {
                        const float4 f = pairs_float4(a, b);
                        uint16_t *out = static_cast<uint16_t *>(args.out[k]) + (int64_t)(y + lane) * cols + x;
                        *reinterpret_cast<uint2 *>(out) = make_uint2(pack(f.x, f.y, f16), pack(f.z, f.w, f16));
                    };
                    const f32x2 a = pair2(s[0]), b = pair2(s[0] + 2);
                    if constexpr (MODE == kGate) {
                        const f32x2 a3 = pair2(s[1]), b3 = pair2(s[1] + 2);
                        f32x2 h[2], g1[2], g3[2];
                        if (args.act == MOE_ACT_SILU) {
                            activate<false, true>(a, a3, h[0], g1[0], g3[0]);
                            activate<false, true>(b, b3, h[1], g1[1], g3[1]);
                        } else {
                            activate<true, true>(a, a3, h[0], g1[0], g3[0]);
                            activate<true, true>(b, b3, h[1], g1[1], g3[1]);
                        }
                        store(0, h[0], h[1]);
                        if (args.f1 != nullptr) {
                            *saved(args.f1) = pairs_float4(g1[0], g1[1]);
                            *saved(args.f3) = pairs_float4(g3[0], g3[1]);
                        }
                    } else if constexpr (MODE == kDHid) {
                        store(0, mul2(a, pair2(&f1.x)), mul2(b, pair2(&f1.z)));
                        store(1, mul2(a, pair2(&f3.x)), mul2(b, pair2(&f3.z)));
                    } else if constexpr (MODE == kLinear) {
                        float e[4];  // (no residual: zeros)
                        if (f16) {
                            unpack2<__half>(res.x, e[0], e[1]);
                            unpack2<__half>(res.y, e[2], e[3]);
                        } else {
                            unpack2<__nv_bfloat16>(res.x, e[0], e[1]);
                            unpack2<__nv_bfloat16>(res.y, e[2], e[3]);
                        }
                        const f32x2 r[2] = {pair2(e), pair2(e + 2)};
                        with_act([&](auto act, auto saves) {
                            f32x2 f[2], df[2];
                            activate_one<act(), saves()>(add2(a, bias[0]), f[0], df[0]);
                            activate_one<act(), saves()>(add2(b, bias[1]), f[1], df[1]);
                            store(0, add2(f[0], r[0]), add2(f[1], r[1]));
                            if (saves()) *saved(args.f1) = pairs_float4(df[0], df[1]);
                        });
                    } else {
                        store(un.p, a, b);
                    }
                }
                __syncwarp();
            }
        };

        // the pair's segment and its join, then the whole tiles
        for (Work w(args, pair, pairs); w.step(); ++uc) {
            const uint32_t a = uc & 1u;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * BN;
            const Unit un = unit_at(w.u);
            auto filled = [&] {
                if (!bounded_wait(ptx::smem_addr(&ctl->tfull[a]), (uc >> 1) & 1u, args.err)) return false;
                ptx::tc_fence_after();
                return true;
            };
            auto release = [&] {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(tempty0 + a * (uint32_t)sizeof(uint64_t));
            };
            if (!w.cut) {
                if (!finish(un, c_lo, c_lo + NC, taddr, false, filled, release)) break;
                continue;
            }
            if (!filled()) break;
            uint32_t *ticket = args.ticket + ((int64_t)w.u * 2 + rank) * kEpiWarps + ew;
            const int j = (pair + share) % args.split;
            const bool few = args.split <= kFewSegments;
            const int step = few ? 8 : 1;  // units of its share come in boxes of 8, or singly
            const int lo = NU / step * j / args.split * step, hi = NU / step * (j + 1) / args.split * step;
            float4 *mine = part_of(pair);
            if (un.row0 + q * 32 >= args.rows[un.p]) {  // nothing to join, in any of its segments
                release();
                continue;
            }
#pragma unroll 1
            for (int v0 = 0; v0 < M * NU; v0 += 8) {
                uint32_t r[32];
                ptx::tmem_ld32(taddr + column(v0), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int u = (v0 + i) % NU;
                    if (u < lo || u >= hi) __stcg(mine + (v0 + i) * 32, words_float4(r + 4 * i));
                }
            }
            __threadfence();
            __syncwarp();
            // low half: parts written; high half: holders that need them no more (one with
            // no units needs none of them)
            if (lane == 0) atomicAdd(ticket, hi > lo ? 1u : 0x10001u);
            if (hi > lo) {
                auto joinable = [&] {
                    bool all = true;
                    if (lane == 0) all = word_wait(ticket, 0xffffu, (uint32_t)args.split, args.err);
                    all = __shfl_sync(0xffffffffu, all, 0) != 0;
                    __syncwarp();  // lane 0's acquire comes before every lane's loads (a shuffle orders none)
                    return all;
                };
                if (few) {
                    if (!finish(un, c_lo + lo / 8, c_lo + hi / 8, taddr, true, joinable, [] {})) break;
                } else {
                    if (!joinable()) break;
                    join(un, taddr, lo, hi);
                }
                // every lane has its parts; the last holder returns the ticket to zero
                __syncwarp();
                if (lane == 0 && atomicAdd(ticket, 0x10000u) >> 16 == (uint32_t)(args.split - 1))
                    *ticket = 0;
            }
            release();
        }
        if (lane == 0) ptx::bulk_wait_group<0>();
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // no arrival or MMA of the pair is outstanding
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc_pair(tmem_base, 2 * BN);
}

// ------------------------------------------------------------ host side --

// Which of `units` tiles of kb k-blocks are cut over `pairs` SM pairs: those past the
// last whole wave, where that is worth a join (about 5 us, the time of kJoin k-blocks,
// for the 256 x 256 sums of each pair to go through L2 and for a launch that starts in
// plain order). At least kMinRun k-blocks a segment. (Over 18 shapes of 66 to 2048
// tokens, inference / training step: kJoin 8 30.7 / 88.6 us, 14 30.4 / 87.8, 18 29.8 /
// 86.8, 26 and more slower again; nothing cut 32.7 / 94.7; a cost for each further
// segment or another kMinRun gained on no average.)
constexpr int kJoin = 18, kMinRun = 8;
void split_work(int64_t units, int kb, int pairs, int *cut, int *split) {
    *cut = *split = 0;
    const int64_t rest = units % pairs;
    if (rest == 0) return;
    const int s = (int)std::min<int64_t>(pairs / rest, kb / kMinRun);
    if (s < 2 || (kb + s - 1) / s + kJoin >= kb) return;
    *cut = (int)rest;
    *split = s;
}

int64_t tiles_of(int rows, int cols, bool gate) {
    const int k = gate ? BN / 2 : BN;
    return (int64_t)((rows + 2 * BM - 1) / (2 * BM)) * ((cols + k - 1) / k);
}

template <int MODE>
cudaError_t launch(const Maps &maps, Args args, cudaStream_t s) {
    const int problems = MODE == kWGrad ? 3 : MODE == kBoth ? 2 : 1;
    int64_t units = 0;
    for (int p = 0; p < 3; ++p) {
        args.first[p] = (int)units;
        if (p >= problems) continue;
        constexpr int kCols = MODE == kGate ? BN / 2 : BN;
        args.mt[p] = (args.rows[p] + 2 * BM - 1) / (2 * BM);
        args.nb[p] = (args.cols[p] + kCols - 1) / kCols;
        units += tiles_of(args.rows[p], args.cols[p], MODE == kGate);
    }
    if (units > (1 << 30)) return cudaErrorInvalidValue;
    args.units = (int)units;
    const int all = std::max(1, std::min(sm_count(), kFfnMaxCtas) / 2);
    if (MODE != kBoth) split_work(units, args.kb, all, &args.cut, &args.split);
    const int pairs = (int)std::min<int64_t>(all, std::max<int64_t>(units, args.cut * args.split));
    args.idesc = idesc(args.f16 != 0, 2 * BM, BN, MODE == kWGrad, !(MODE == kDHid || MODE == kDX || MODE == kBoth));
    args.idesc_dw = idesc(args.f16 != 0, 2 * BM, BN, true, true);
    const cudaError_t e =
        ensure_dynamic_smem(reinterpret_cast<const void *>(dense_gemm_kernel<MODE>), (int)kSmem);
    if (e != cudaSuccess) return e;
    if (args.cut > 0)
        return launch_together(dense_gemm_kernel<MODE>, dim3(2 * pairs), dim3(kThreads), kSmem, s, maps, args);
    return launch_k(dense_gemm_kernel<MODE>, dim3(2 * pairs), dim3(kThreads), kSmem, s, maps, args);
}

// Whether dX [T,k] and dW [k,n] of a projection run in one launch: where their tiles fit the
// SM pairs together and the longer reduction takes less than both launches (in k-blocks, with a
// launch's start, fill and end as kStart). The whole backward, two launches against one: 777 x
// 1000 x 2728 35.0 / 27.0 us, 2432 x 560 x 256 24.7 / 22.2, 375 x 424 x 656 19.0 / 12.3; where the
// reductions are too long for tiles that are not cut, and two launches stay: 70 x 576 x 3864 26.3 /
// 29.7, 256 x 256 x 8192 28.8 / 56.3.
constexpr int kStart = 18;
int64_t launch_blocks(int64_t units, int kb, int pairs) {
    int cut, split;
    split_work(units, kb, pairs, &cut, &split);
    const int64_t whole = (units - cut + pairs - 1) / pairs * kb;
    return kStart + std::max<int64_t>(whole, cut > 0 ? (kb + split - 1) / split + kJoin : 0);
}
bool both_in_one(int T, int k, int n, int pairs) {
    const int64_t x = tiles_of(T, k, false), w = tiles_of(k, n, false);
    const int kx = (n + BK - 1) / BK, kw = (T + BK - 1) / BK;
    return x + w <= pairs && kStart + std::max(kx, kw) < launch_blocks(x, kx, pairs) + launch_blocks(w, kw, pairs);
}

constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B, kSw64 = CU_TENSOR_MAP_SWIZZLE_64B;

// Operand maps: K-major A rows (64 x 128 boxes) and 64 x 64 boxes for the rest.
bool map_a(CUtensorMap *m, bool f16, const void *p, int cols, int rows) {
    return make_map(m, map_type(f16), p, cols, rows, 64, BM, kSw128);
}
bool map_64(CUtensorMap *m, bool f16, const void *p, int cols, int rows) {
    return make_map(m, map_type(f16), p, cols, rows, 64, 64, kSw128);
}
bool map_out(CUtensorMap *m, bool f16, const void *p, int cols, int rows) {
    return make_map(m, map_type(f16), p, cols, rows, 32, 32, kSw64);
}

}  // namespace
}  // namespace ffn

using namespace ffn;

size_t ffn_dense_part_bytes() {
    // a segment for each pair (which products are cut depends on the device's SMs)
    return (size_t)kFfnMaxCtas * kEpiWarps * kPartVecs * sizeof(float4);
}

cudaError_t launch_ffn_gate(const void *X, const void *W1, const void *W3, int T, int d, int n,
                            int act, bool f16, void *H, float *F1, float *F3, float4 *part,
                            uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    Maps m{};
    if (!map_a(&m.a[0], f16, X, d, T) || !map_64(&m.b[0], f16, W1, n, d) ||
        !map_64(&m.b[1], f16, W3, n, d) || !map_out(&m.o[0], f16, H, n, T))
        return cudaErrorInvalidValue;
    Args a{};
    a.rows[0] = T;
    a.cols[0] = n;
    a.kb = (d + BK - 1) / BK;
    a.f16 = f16;
    a.act = act;
    a.out[0] = H;
    a.f1 = F1;
    a.f3 = F3;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    return launch<kGate>(m, a, s);
}

cudaError_t launch_ffn_down(const void *H, const void *W2, int T, int d, int n, bool f16, void *Y,
                            float4 *part, uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    Maps m{};
    if (!map_a(&m.a[0], f16, H, n, T) || !map_64(&m.b[0], f16, W2, d, n) ||
        !map_out(&m.o[0], f16, Y, d, T))
        return cudaErrorInvalidValue;
    Args a{};
    a.rows[0] = T;
    a.cols[0] = d;
    a.kb = (n + BK - 1) / BK;
    a.f16 = f16;
    a.out[0] = Y;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    return launch<kDown>(m, a, s);
}

cudaError_t launch_linear_tiled(const LinearCall &c, float *F, float4 *part, uint32_t *ticket, uint32_t *err,
                                cudaStream_t s) {
    Maps m{};
    if (!map_a(&m.a[0], c.f16, c.X, c.k, c.T) || !map_64(&m.b[0], c.f16, c.W, c.n, c.k) ||
        !map_out(&m.o[0], c.f16, c.Y, c.n, c.T))
        return cudaErrorInvalidValue;
    Args a{};
    a.rows[0] = c.T;
    a.cols[0] = c.n;
    a.kb = (c.k + BK - 1) / BK;
    a.f16 = c.f16;
    a.act = c.act;
    a.bias = c.bias;
    a.bias32 = c.bias32;
    a.res = c.res;
    a.f1 = F;
    a.out[0] = c.Y;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    return launch<kLinear>(m, a, s);
}

cudaError_t launch_linear_products(const void *dA, const void *X, const void *W, int T, int k, int n, bool f16,
                                   void *dX, void *dW, void *dbias, bool bias32, const float *sums,
                                   float4 *part, uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    Maps m{};
    Args a{};
    a.f16 = f16;
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    a.dbias = dbias;
    a.bias32 = bias32;
    a.sums = sums;
    a.sum_rows = linear_sum_rows(T, n);
    a.sum_n = n;
    const int kx = (n + BK - 1) / BK, kw = (T + BK - 1) / BK;
    if (dX != nullptr && dW != nullptr && both_in_one(T, k, n, sm_count() / 2)) {
        if (!map_a(&m.a[0], f16, dA, n, T) || !map_64(&m.b[0], f16, W, n, k) || !map_out(&m.o[0], f16, dX, k, T) ||
            !map_64(&m.a[1], f16, X, k, T) || !map_64(&m.b[1], f16, dA, n, T) || !map_out(&m.o[1], f16, dW, n, k))
            return cudaErrorInvalidValue;
        a.rows[0] = T;
        a.cols[0] = a.rows[1] = k;
        a.cols[1] = n;
        a.kb = kx;
        a.kb_dw = kw;
        a.out[0] = dX;
        a.out[1] = dW;
        return launch<kBoth>(m, a, s);
    }
    if (dX != nullptr) {
        if (!map_a(&m.a[0], f16, dA, n, T) || !map_64(&m.b[0], f16, W, n, k) || !map_out(&m.o[0], f16, dX, k, T))
            return cudaErrorInvalidValue;
        m.a[1] = m.a[0];
        m.b[1] = m.b[0];
        a.rows[0] = T;
        a.cols[0] = k;
        a.kb = a.kb_half = kx;
        a.out[0] = dX;
        const cudaError_t e = launch<kDX>(m, a, s);
        if (e != cudaSuccess) return e;
    }
    if (dW == nullptr) return cudaSuccess;
    if (!map_64(&m.a[0], f16, X, k, T) || !map_64(&m.b[0], f16, dA, n, T) || !map_out(&m.o[0], f16, dW, n, k))
        return cudaErrorInvalidValue;
    for (int i = 1; i < 3; ++i) {  // one problem of three
        m.a[i] = m.a[0];
        m.b[i] = m.b[0];
        m.o[i] = m.o[0];
    }
    a.rows[0] = k;
    a.cols[0] = n;
    a.kb = kw;
    a.out[0] = dW;
    return launch<kWGrad>(m, a, s);
}

cudaError_t launch_ffn_backward(const void *dY, const void *X, const void *W1, const void *W3,
                                const void *W2, const void *H, const float *F1, const float *F3,
                                int T, int d, int n, bool f16, void *dA1, void *dA3,
                                void *dX, void *dW1, void *dW3, void *dW2, float4 *part,
                                uint32_t *ticket, uint32_t *err, cudaStream_t s) {
    Maps m{};
    if (!map_a(&m.a[0], f16, dY, d, T) || !map_64(&m.b[0], f16, W2, d, n) ||
        !map_out(&m.o[0], f16, dA1, n, T) || !map_out(&m.o[1], f16, dA3, n, T))
        return cudaErrorInvalidValue;
    Args a{};
    a.rows[0] = T;
    a.cols[0] = n;
    a.kb = (d + BK - 1) / BK;
    a.f16 = f16;
    a.out[0] = dA1;
    a.out[1] = dA3;
    a.f1 = const_cast<float *>(F1);
    a.f3 = const_cast<float *>(F3);
    a.part = part;
    a.ticket = ticket;
    a.err = err;
    cudaError_t e = launch<kDHid>(m, a, s);
    if (e != cudaSuccess) return e;
    if (dX != nullptr) {
        if (!map_a(&m.a[0], f16, dA1, n, T) || !map_a(&m.a[1], f16, dA3, n, T) ||
            !map_64(&m.b[0], f16, W1, n, d) || !map_64(&m.b[1], f16, W3, n, d) ||
            !map_out(&m.o[0], f16, dX, d, T))
            return cudaErrorInvalidValue;
        a.cols[0] = d;
        a.kb_half = (n + BK - 1) / BK;
        a.kb = 2 * a.kb_half;
        a.out[0] = dX;
        if ((e = launch<kDX>(m, a, s)) != cudaSuccess) return e;
    }
    if (dW1 == nullptr) return cudaSuccess;
    if (!map_64(&m.a[0], f16, X, d, T) || !map_64(&m.a[1], f16, X, d, T) ||
        !map_64(&m.a[2], f16, H, n, T) || !map_64(&m.b[0], f16, dA1, n, T) ||
        !map_64(&m.b[1], f16, dA3, n, T) || !map_64(&m.b[2], f16, dY, d, T) ||
        !map_out(&m.o[0], f16, dW1, n, d) || !map_out(&m.o[1], f16, dW3, n, d) ||
        !map_out(&m.o[2], f16, dW2, d, n))
        return cudaErrorInvalidValue;
    a.rows[0] = a.rows[1] = a.cols[2] = d;
    a.cols[0] = a.cols[1] = a.rows[2] = n;
    a.kb = (T + BK - 1) / BK;
    a.out[0] = dW1;
    a.out[1] = dW3;
    a.out[2] = dW2;
    return launch<kWGrad>(m, a, s);
}

}  // namespace moe
