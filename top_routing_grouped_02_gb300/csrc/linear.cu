// What a projection's gradients need beside the products of ffn.cu: dA = dY F, F = act'(A),
// rounded to 16 bits as the tensor cores' operand, and the bias' gradient, the sums over rows
// of dY F before that rounding. The rounding is all that dX and dW lose but for their own: for bf16
// they are 2.35e-3 off in the 2-norm where one rounding is 1.66e-3. (dA as the sum of two 16-bit
// matrices would keep them at that, for twice the products: 504 us more of a 970 us step at 4096 x 4096 x 14336.)
//
// Bound by HBM: dY (16 bits) and F (fp32, in blocks of 32 x 32, the columns by fours: see
// moe_ffn_forward_train) are read once and dA is written once, in the same pass as the sums. A
// block of 8 warps takes 256 columns of its run of rows, 32 rows at a time. A warp's lanes are 8
// rows x 4 groups of 8 columns: its loads of F are 128 consecutive bytes for each group, those
// of dY 64 for each row, and the neighbouring warps take the rest of the rows' lines. Each
// thread sums its columns over its rows, the 8 lanes of a column are added by shuffles and the
// blocks' partial rows in order by the weight gradient's launch or (without it, or many of them) a kernel
// of their own: the result does not depend on timing.
// Measured: 4096 x 14336 bf16 71 us (6.6 TB/s), 777 x 2728 6 us.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kCols = 32 * kWarps;  // of a block
constexpr int kRows = 32;                       // at a time: four of each lane's in flight

constexpr int kBlocks = 8 * 152;

template <typename T, bool FACTOR>
__global__ void __launch_bounds__(32 * kWarps)
linear_grad_kernel(const T *dY, const float *F, int rows, int n, T *dA, float *sums) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const int block = blockIdx.x * kWarps + warp;  // of 32 columns
    const int col = block * 32 + (lane >> 3) * 8;
    const int groups = (rows + kRows - 1) / kRows;
    const int g0 = (int)((int64_t)groups * blockIdx.y / gridDim.y);
    const int g1 = (int)((int64_t)groups * (blockIdx.y + 1) / gridDim.y);
    float s[8] = {};
    if (col < n) {  // n is a multiple of 8
        for (int g = g0; g < g1; ++g) {
            const int64_t at = (int64_t)(g * kRows + sub) * n + col;
            uint4 y[4];
            float4 f[4][2];
            const float4 *from = reinterpret_cast<const float4 *>(F) +
                                 ((int64_t)g * ((n + 31) / 32) + block) * 256 + (lane >> 3) * 64 + sub;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (g * kRows + sub + 8 * k >= rows) continue;
                y[k] = *reinterpret_cast<const uint4 *>(dY + at + (int64_t)8 * k * n);
                if (FACTOR) {
                    f[k][0] = __ldcs(from + 8 * k);
                    f[k][1] = __ldcs(from + 8 * k + 32);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (g * kRows + sub + 8 * k >= rows) continue;
                float v[8];
                to_f32<T, 8>(y[k], v);
                if (FACTOR) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= (&f[k][j >> 2].x)[j & 3];
                    *reinterpret_cast<uint4 *>(dA + at + (int64_t)8 * k * n) = from_f32<T, 8>(v);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] += v[j];
            }
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int o = 1; o < 8; o *= 2)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    if (sub == 0 && col < n) {
        float4 *out = reinterpret_cast<float4 *>(sums + (int64_t)blockIdx.y * n + col);
        out[0] = make_float4(s[0], s[1], s[2], s[3]);
        out[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
}

template <typename T>
cudaError_t launch_grad(const void *dY, const float *F, int rows, int n, void *dA, float *sums, cudaStream_t s) {
    const dim3 grid((n + kCols - 1) / kCols, linear_sum_rows(rows, n)), block(32 * kWarps);
    const T *y = static_cast<const T *>(dY);
    return F != nullptr ? launch_k(linear_grad_kernel<T, true>, grid, block, 0, s, y, F, rows, n,
                                   static_cast<T *>(dA), sums)
                        : launch_k(linear_grad_kernel<T, false>, grid, block, 0, s, y, F, rows, n,
                                   static_cast<T *>(nullptr), sums);
}

}  // namespace

// Blocks over the rows: as many as make eight for each SM of the device (a constant: a
// workspace's size does not depend on the device at hand).
int linear_sum_rows(int T, int n) {
    const int64_t across = (n + kCols - 1) / kCols, most = ((int64_t)T + kRows - 1) / kRows;
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kBlocks / across));
}

cudaError_t launch_linear_grad(const void *dY, const float *F, int T, int n, bool f16, void *dA, float *sums,
                               cudaStream_t s) {
    if (F == nullptr && sums == nullptr) return cudaSuccess;
    return f16 ? launch_grad<__half>(dY, F, T, n, dA, sums, s) : launch_grad<__nv_bfloat16>(dY, F, T, n, dA, sums, s);
}

cudaError_t launch_linear_bias(const float *sums, int T, int n, bool f16, void *dbias, bool bias32, cudaStream_t s) {
    // (n is even: a row of sums is two halves, as the reduction takes them)
    const moe_dtype_t wt = bias32 ? MOE_DTYPE_F32 : f16 ? MOE_DTYPE_F16 : MOE_DTYPE_BF16;
    return launch_weight_reduce(sums, linear_sum_rows(T, n), n / 2, wt, dbias,
                                static_cast<char *>(dbias) + (size_t)(n / 2) * (bias32 ? 4 : 2), s);
}

}  // namespace moe
