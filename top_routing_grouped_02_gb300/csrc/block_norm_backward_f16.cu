#include "block_norm_backward.cuh"

namespace moe {
namespace bn {
template cudaError_t backward_type<__half>(const Args &, int, int *, cudaStream_t);
}  // namespace bn
}  // namespace moe
