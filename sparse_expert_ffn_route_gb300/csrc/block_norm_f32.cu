// block_norm_f32.cu -- the norms' launches for a stream in fp32.
#include "block_norm_launch.cuh"

namespace moe {
namespace norm {

template cudaError_t launch_forward<float>(const NormArgs &p, int dtype, cudaStream_t st);
template cudaError_t launch_backward<float>(NormArgs p, int dtype, int parts, cudaStream_t st);

}  // namespace norm
}  // namespace moe
