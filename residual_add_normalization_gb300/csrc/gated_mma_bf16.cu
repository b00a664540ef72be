// The gated product on the tensor cores, bfloat16.
#include "linear_mma_launch.cuh"

namespace b200norm {

template cudaError_t launch_mma_gated_t<__nv_bfloat16>(const Product&, const MmaPlan&, int,
                                                       unsigned*, cudaStream_t);

}  // namespace b200norm
