// Shared by the kernels of the dense gated feed-forward block: tensor maps,
// bounded barrier waits, the activations and 16-bit packing.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "elem.cuh"
#include "ptx.cuh"

namespace moe {
namespace ffn {

// 2-D tensor [rows, cols] of 16-bit (bf16 or fp16) or fp32 elements, cols
// contiguous, rows dense; loads fill zeros and stores write nothing outside it.
bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols,
              uint64_t rows, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle);
inline CUtensorMapDataType map_type(bool f16) {
    return f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

constexpr uint64_t kWaitLimitNs = 1000000000ull;

// Polls a barrier of this CTA; after about one second it sets MOE_DEVERR_TIMEOUT
// and gives up. (The clock comes before the last look: a block that was itself held up for
// longer does not give up on what has arrived meanwhile.)
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, uint32_t *err) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        const bool late = (spin & 63u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs;
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (late) {
            atomicOr(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Polls a word in global memory (acquire) until done(word), bounded like bounded_wait.
template <typename Done>
__device__ __forceinline__ bool poll_word(const uint32_t *w, uint32_t *err, Done done) {
    if (done(ptx::ld_acquire_gpu(w))) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        __nanosleep(32);
        const bool late = (spin & 15u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs;
        if (done(ptx::ld_acquire_gpu(w))) return true;
        if (late) {
            atomicOr(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
    }
}
// Until (word & mask) == want; until word >= least.
__device__ __forceinline__ bool word_wait(const uint32_t *w, uint32_t mask, uint32_t want,
                                          uint32_t *err) {
    return poll_word(w, err, [=](uint32_t v) { return (v & mask) == want; });
}
__device__ __forceinline__ bool word_wait_least(const uint32_t *w, uint32_t least, uint32_t *err) {
    return poll_word(w, err, [=](uint32_t v) { return v >= least; });
}

// Four columns.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
}

// Both activations are a * sigmoid(z(a)): SiLU with z = a, GELU's tanh form
// 0.5 a (1 + tanh(u)) = a sigmoid(2 u) with z = 2 u = k (a + 0.044715 a^3),
// k = 2 sqrt(2 / pi). sg: the sigmoid.
__device__ __forceinline__ float act_sigmoid(float a, int act) {
    const float z = act == MOE_ACT_SILU ? a : 1.5957691216f * fmaf(0.044715f * a * a, a, a);
    return __fdividef(1.0f, 1.0f + __expf(-z));
}
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
// For a pair of elements: h = act(a1) a3, f3 = act(a1) and (TRAIN) f1 = a3 act'(a1),
//   act' = sg + a sg (1 - sg) z'(a).
// Packed, with the sigmoid as 1 / (1 + 2^(-z log2 e)) and the branch on the activation
// outside: an epilogue whose tile has a short reduction is bound by its instructions.
template <bool GELU, bool TRAIN>
__device__ __forceinline__ void activate(f32x2 a1, f32x2 a3, f32x2 &h, f32x2 &f1, f32x2 &f3) {
    constexpr float kLog2e = 1.44269504f, kZ = 1.5957691216f, kCube = 0.044715f;
    f32x2 t, sq = 0;
    if (GELU) {
        sq = mul2(a1, a1);
        t = mul2(a1, fma2(sq, both(-kLog2e * kZ * kCube), both(-kLog2e * kZ)));
    } else {
        t = mul2(a1, both(-kLog2e));
    }
    float x, y;
    unpair(t, x, y);
    unpair(add2(pair(exp2_approx(x), exp2_approx(y)), both(1.f)), x, y);
    const f32x2 sg = pair(rcp_approx(x), rcp_approx(y));
    f3 = mul2(a1, sg);
    h = mul2(f3, a3);
    if (TRAIN) {
        f32x2 u = fma2(sg, both(-1.f), both(1.f));
        if (GELU) u = mul2(u, fma2(sq, both(3.f * kZ * kCube), both(kZ)));
        f1 = mul2(a3, fma2(f3, u, sg));
    }
}

// A projection's activation of a pair, f = act(a), and (TRAIN) df = act'(a). ACT: moe_act_t, or
// kNoAct: f = a.
constexpr int kNoAct = MOE_ACT_NONE;
template <int ACT, bool TRAIN>
__device__ __forceinline__ void activate_one(f32x2 a, f32x2 &f, f32x2 &df) {
    if constexpr (ACT == kNoAct) {
        f = a;
        if (TRAIN) df = both(1.f);
    } else {
        f32x2 h;
        activate<ACT == MOE_ACT_GELU_TANH, TRAIN>(a, both(1.f), h, df, f);
    }
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, bool f16) {
    return f16 ? pack2<__half>(lo, hi) : pack2<__nv_bfloat16>(lo, hi);
}
__device__ __forceinline__ uint16_t round16(float v, bool f16) {
    return (uint16_t)(pack(v, 0.f, f16) & 0xffffu);
}

// Element i of a 16-bit vector.
__device__ __forceinline__ float load16(const void *p, int64_t i, bool f16) {
    const uint32_t w = static_cast<const uint16_t *>(p)[i];
    float x, unused;
    if (f16) unpack2<__half>(w, x, unused);
    else unpack2<__nv_bfloat16>(w, x, unused);
    return x;
}

// Instruction descriptor: fp32 accumulator, A and B both bf16 or both fp16.
constexpr uint32_t idesc(bool f16, int M, int N, bool a_mn, bool b_mn) {
    return f16 ? ptx::idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10))
               : ptx::idesc_bf16(M, N, a_mn, b_mn);
}

}  // namespace ffn
}  // namespace moe
