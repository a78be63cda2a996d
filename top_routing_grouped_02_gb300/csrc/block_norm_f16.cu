#include "block_norm_forward.cuh"

namespace moe {
namespace bn {
template cudaError_t forward_type<__half>(const Args &, int, cudaStream_t);
}  // namespace bn
}  // namespace moe
