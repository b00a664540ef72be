// The gated product on the tensor cores, float16.
#include "linear_mma_launch.cuh"

namespace b200norm {

template cudaError_t launch_mma_gated_t<__half>(const Product&, const MmaPlan&, int, unsigned*,
                                             cudaStream_t);

}  // namespace b200norm
