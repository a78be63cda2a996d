// Element types of the sub-block operators (norms, dropout, dispatch and combine, dense block and
// projections): packed pairs and vectors of V elements as one raw register value, converted to and from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> { using type = uint4; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<2> { using type = uint16_t; };

template <typename T, int V>
using Raw = typename RawOf<sizeof(T) * V>::type;

// 16-bit pairs packed in a word: element 0 in the low half.
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float &a, float &b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t w, float &a, float &b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// V elements of a raw value as fp32, and back (each element rounded once, to
// nearest even).
template <typename T, int V>
__device__ __forceinline__ void to_f32(const Raw<T, V> &r, float *f) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4) {
            f[0] = __uint_as_float(r.x);
            f[1] = __uint_as_float(r.y);
            f[2] = __uint_as_float(r.z);
            f[3] = __uint_as_float(r.w);
        } else if constexpr (V == 2) {
            f[0] = __uint_as_float(r.x);
            f[1] = __uint_as_float(r.y);
        } else {
            f[0] = __uint_as_float(r);
        }
    } else if constexpr (V == 8) {
        unpack2<T>(r.x, f[0], f[1]);
        unpack2<T>(r.y, f[2], f[3]);
        unpack2<T>(r.z, f[4], f[5]);
        unpack2<T>(r.w, f[6], f[7]);
    } else if constexpr (V == 4) {
        unpack2<T>(r.x, f[0], f[1]);
        unpack2<T>(r.y, f[2], f[3]);
    } else if constexpr (V == 2) {
        unpack2<T>(r, f[0], f[1]);
    } else {
        float unused;
        unpack2<T>((uint32_t)r, f[0], unused);
    }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> from_f32(const float *f) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4)
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
        else if constexpr (V == 2)
            return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
        else
            return __float_as_uint(f[0]);
    } else if constexpr (V == 8) {
        return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                          pack2<T>(f[6], f[7]));
    } else if constexpr (V == 4) {
        return make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
    } else if constexpr (V == 2) {
        return pack2<T>(f[0], f[1]);
    } else {
        return (uint16_t)(pack2<T>(f[0], 0.f) & 0xffffu);
    }
}

// Pairs of fp32 values in one 64-bit register: the packed arithmetic of sm_100 and
// later does two operations an instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ void unpair(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float pair_sum(f32x2 v) {
    float lo, hi;
    unpair(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// A 16-byte vector of V elements as V / 2 pairs, and back.
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const uint4 &r, f32x2 *p) {
    float f[V];
    to_f32<T, V>(r, f);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) p[j] = pair(f[2 * j], f[2 * j + 1]);
}
template <typename T, int V>
__device__ __forceinline__ uint4 from_pairs(const f32x2 *p) {
    float f[V];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) unpair(p[j], f[2 * j], f[2 * j + 1]);
    return from_f32<T, V>(f);
}

template <typename T>
__device__ __forceinline__ float load_f32(const T *p) { return (float)*p; }
template <typename T>
__device__ __forceinline__ void store_f32(T *p, float v) {
    if constexpr (sizeof(T) == 4) *p = v;
    else if constexpr (sizeof(T) == 2) *reinterpret_cast<uint16_t *>(p) = (uint16_t)(pack2<T>(v, 0.f) & 0xffffu);
}

}  // namespace moe
