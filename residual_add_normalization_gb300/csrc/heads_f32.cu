// The head kernels, float32.
#include "heads_launch.cuh"

namespace b200norm {

template cudaError_t launch_heads_t<float>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_grad_t<float>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_dgamma_t<float>(const HeadsCall&, HeadParts, cudaStream_t);

}  // namespace b200norm
