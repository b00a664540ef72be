// Layer normalization, bfloat16 rows with bfloat16 or float32 gamma and beta.
#include "layer_launch.cuh"

namespace b200norm {

template cudaError_t launch_layer_tm<__nv_bfloat16, __nv_bfloat16>(const LayerCall&, cudaStream_t);
template cudaError_t launch_layer_tm<__nv_bfloat16, float>(const LayerCall&, cudaStream_t);
template cudaError_t launch_layer_grad_tm<__nv_bfloat16, __nv_bfloat16>(const LayerGradCall&, cudaStream_t);
template cudaError_t launch_layer_grad_tm<__nv_bfloat16, float>(const LayerGradCall&, cudaStream_t);

}  // namespace b200norm
