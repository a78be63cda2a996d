#include "block_norm_backward.cuh"

namespace moe {
namespace bn {
template cudaError_t backward_type<float>(const Args &, int, int *, cudaStream_t);
}  // namespace bn
}  // namespace moe
