// The linear operator without the tensor cores, float32.
#include "linear_launch.cuh"

namespace b200norm {

cudaError_t launch_plain_f32(const Product& p, cudaStream_t stream) { return launch_plain(p, stream); }

template cudaError_t launch_rows<float>(const Product&, cudaStream_t);
template cudaError_t launch_dz<float>(const LinearDzCall&, cudaStream_t);

}  // namespace b200norm
