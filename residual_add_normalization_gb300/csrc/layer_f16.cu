// Layer normalization, float16 rows with float16 or float32 gamma and beta.
#include "layer_launch.cuh"

namespace b200norm {

template cudaError_t launch_layer_tm<__half, __half>(const LayerCall&, cudaStream_t);
template cudaError_t launch_layer_tm<__half, float>(const LayerCall&, cudaStream_t);
template cudaError_t launch_layer_grad_tm<__half, __half>(const LayerGradCall&, cudaStream_t);
template cudaError_t launch_layer_grad_tm<__half, float>(const LayerGradCall&, cudaStream_t);

}  // namespace b200norm
