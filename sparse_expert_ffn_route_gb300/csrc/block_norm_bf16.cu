// block_norm_bf16.cu -- the norms' launches for a stream in bf16.
#include "block_norm_launch.cuh"

namespace moe {
namespace norm {

template cudaError_t launch_forward<__nv_bfloat16>(const NormArgs &p, int dtype, cudaStream_t st);
template cudaError_t launch_backward<__nv_bfloat16>(NormArgs p, int dtype, int parts, cudaStream_t st);

}  // namespace norm
}  // namespace moe
