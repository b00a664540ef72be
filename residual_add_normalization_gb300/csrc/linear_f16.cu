// The linear operator without the tensor cores, float16.
#include "gated_few.cuh"
#include "linear_launch.cuh"

namespace b200norm {

template cudaError_t launch_rows<__half>(const Product&, cudaStream_t);
template cudaError_t launch_dz<__half>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_gated_dz<__half>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_db<__half>(const LinearDzCall&, bool, bool, cudaStream_t);
template cudaError_t launch_gated_few<__half>(const GatedFewArgs&, void*, cudaStream_t);
template cudaError_t launch_pack<__half>(const void*, void*, int64_t, const void*, void*, int64_t,
                               int64_t, cudaStream_t);

}  // namespace b200norm
