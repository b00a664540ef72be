// The head kernels, float16.
#include "heads_launch.cuh"

namespace b200norm {

template cudaError_t launch_heads_t<__half>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_grad_t<__half>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_dgamma_t<__half>(const HeadsCall&, HeadParts, cudaStream_t);

}  // namespace b200norm
