#include "block_norm_forward.cuh"

namespace moe {
namespace bn {
template cudaError_t forward_type<__nv_bfloat16>(const Args &, int, cudaStream_t);
}  // namespace bn
}  // namespace moe
