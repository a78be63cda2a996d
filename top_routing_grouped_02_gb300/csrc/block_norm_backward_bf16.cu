#include "block_norm_backward.cuh"

namespace moe {
namespace bn {
template cudaError_t backward_type<__nv_bfloat16>(const Args &, int, int *, cudaStream_t);
}  // namespace bn
}  // namespace moe
