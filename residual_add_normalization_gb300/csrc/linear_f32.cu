// The linear operator without the tensor cores, float32.
#include "linear_launch.cuh"

namespace b200norm {

template cudaError_t launch_plain<float>(const Product&, cudaStream_t);
template cudaError_t launch_rows<float>(const Product&, cudaStream_t);
template cudaError_t launch_dz<float>(const LinearDzCall&, cudaStream_t);

}  // namespace b200norm
