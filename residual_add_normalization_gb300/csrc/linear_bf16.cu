// The linear operator without the tensor cores, bfloat16.
#include "linear_launch.cuh"

namespace b200norm {

template cudaError_t launch_rows<__nv_bfloat16>(const Product&, cudaStream_t);
template cudaError_t launch_dz<__nv_bfloat16>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_pack<__nv_bfloat16>(const void*, void*, int64_t, const void*, void*, int64_t,
                                      int64_t, cudaStream_t);

}  // namespace b200norm
