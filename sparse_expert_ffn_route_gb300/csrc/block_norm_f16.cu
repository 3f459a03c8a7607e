// block_norm_f16.cu -- the norms' launches for a stream in fp16.
#include "block_norm_launch.cuh"

namespace moe {
namespace norm {

template cudaError_t launch_forward<__half>(const NormArgs &p, int dtype, cudaStream_t st);
template cudaError_t launch_backward<__half>(NormArgs p, int dtype, int parts, cudaStream_t st);

}  // namespace norm
}  // namespace moe
