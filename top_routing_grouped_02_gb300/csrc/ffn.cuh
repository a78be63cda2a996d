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
// and gives up.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, uint32_t *err) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((spin & 63u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Polls a word in global memory (acquire) until (word & mask) == want, bounded like
// bounded_wait.
__device__ __forceinline__ bool word_wait(const uint32_t *w, uint32_t mask, uint32_t want,
                                          uint32_t *err) {
    if ((ptx::ld_acquire_gpu(w) & mask) == want) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        __nanosleep(32);
        if ((ptx::ld_acquire_gpu(w) & mask) == want) return true;
        if ((spin & 15u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Both activations are a * sigmoid(z(a)): SiLU with z = a, GELU's tanh form
// 0.5 a (1 + tanh(u)) = a sigmoid(2 u) with z = 2 u = k (a + 0.044715 a^3),
// k = 2 sqrt(2 / pi). sg: the sigmoid.
__device__ __forceinline__ float act_sigmoid(float a, int act) {
    const float z = act == MOE_ACT_SILU ? a : 1.5957691216f * fmaf(0.044715f * a * a, a, a);
    return __fdividef(1.0f, 1.0f + __expf(-z));
}
// Derivative sg + a sg (1 - sg) z'(a).
__device__ __forceinline__ float act_grad(float a, float sg, int act) {
    const float dz = act == MOE_ACT_SILU ? 1.0f : 1.5957691216f * fmaf(3.0f * 0.044715f * a, a, 1.0f);
    return sg * fmaf(a * (1.0f - sg), dz, 1.0f);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, bool f16) {
    return f16 ? pack2<__half>(lo, hi) : pack2<__nv_bfloat16>(lo, hi);
}
__device__ __forceinline__ uint16_t round16(float v, bool f16) {
    return (uint16_t)(pack(v, 0.f, f16) & 0xffffu);
}

// Instruction descriptor: fp32 accumulator, A and B both bf16 or both fp16.
constexpr uint32_t idesc(bool f16, int M, int N, bool a_mn, bool b_mn) {
    return f16 ? ptx::idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10))
               : ptx::idesc_bf16(M, N, a_mn, b_mn);
}

}  // namespace ffn
}  // namespace moe
