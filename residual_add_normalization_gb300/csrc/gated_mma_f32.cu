// The gated product and its gradients' products on the tensor cores, float32 in three bfloat16
// pieces.
#include "linear_mma_launch.cuh"

namespace b200norm {

cudaError_t launch_mma_f32(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                           cudaStream_t stream) {
  if (p.gated) return launch_mma_gated_t<__nv_bfloat16, float>(p, plan, sms, status, stream);
  return p.a.k_contiguous ? launch_mma_pieces<true>(p, plan, sms, status, stream)
                          : launch_mma_pieces<false>(p, plan, sms, status, stream);
}

}  // namespace b200norm
