// The head kernels, bfloat16.
#include "heads_launch.cuh"

namespace b200norm {

template cudaError_t launch_heads_t<__nv_bfloat16>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_grad_t<__nv_bfloat16>(const HeadsCall&, cudaStream_t);
template cudaError_t launch_heads_dgamma_t<__nv_bfloat16>(const HeadsCall&, HeadParts,
                                                          cudaStream_t);

}  // namespace b200norm
