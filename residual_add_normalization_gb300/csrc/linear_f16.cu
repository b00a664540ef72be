// The linear operator without the tensor cores, float16.
#include "linear_launch.cuh"

namespace b200norm {

template cudaError_t launch_rows<__half>(const Product&, cudaStream_t);
template cudaError_t launch_dz<__half>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_pack<__half>(const void*, void*, int64_t, const void*, void*, int64_t,
                               int64_t, cudaStream_t);

}  // namespace b200norm
