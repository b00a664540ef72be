// Layer normalization, float32 rows; and the switch over the (T, M) pairs.
#include <atomic>

#include "layer_launch.cuh"

namespace b200norm {

template cudaError_t launch_layer_tm<float, float>(const LayerCall&, cudaStream_t);
template cudaError_t launch_layer_grad_tm<float, float>(const LayerGradCall&, cudaStream_t);

extern template cudaError_t launch_layer_tm<__half, __half>(const LayerCall&, cudaStream_t);
extern template cudaError_t launch_layer_tm<__half, float>(const LayerCall&, cudaStream_t);
extern template cudaError_t launch_layer_tm<__nv_bfloat16, __nv_bfloat16>(const LayerCall&,
                                                                          cudaStream_t);
extern template cudaError_t launch_layer_tm<__nv_bfloat16, float>(const LayerCall&, cudaStream_t);
extern template cudaError_t launch_layer_grad_tm<__half, __half>(const LayerGradCall&,
                                                                 cudaStream_t);
extern template cudaError_t launch_layer_grad_tm<__half, float>(const LayerGradCall&,
                                                                cudaStream_t);
extern template cudaError_t launch_layer_grad_tm<__nv_bfloat16, __nv_bfloat16>(
    const LayerGradCall&, cudaStream_t);
extern template cudaError_t launch_layer_grad_tm<__nv_bfloat16, float>(const LayerGradCall&,
                                                                       cudaStream_t);

static std::atomic<unsigned long long> g_layer_withhold{0};

unsigned long long layer_withhold_limit_ns() { return g_layer_withhold.load(); }
void set_layer_withhold(unsigned long long limit_ns) { g_layer_withhold.store(limit_ns); }

cudaError_t launch_layer(const LayerCall& c, cudaStream_t stream) {
  const bool m32 = c.m == DType::F32;
  switch (c.t) {
    case DType::F32: return launch_layer_tm<float, float>(c, stream);
    case DType::F16:
      return m32 ? launch_layer_tm<__half, float>(c, stream)
                 : launch_layer_tm<__half, __half>(c, stream);
    default:
      return m32 ? launch_layer_tm<__nv_bfloat16, float>(c, stream)
                 : launch_layer_tm<__nv_bfloat16, __nv_bfloat16>(c, stream);
  }
}

cudaError_t launch_layer_grad(const LayerGradCall& c, cudaStream_t stream) {
  const bool m32 = c.m == DType::F32;
  switch (c.t) {
    case DType::F32: return launch_layer_grad_tm<float, float>(c, stream);
    case DType::F16:
      return m32 ? launch_layer_grad_tm<__half, float>(c, stream)
                 : launch_layer_grad_tm<__half, __half>(c, stream);
    default:
      return m32 ? launch_layer_grad_tm<__nv_bfloat16, float>(c, stream)
                 : launch_layer_grad_tm<__nv_bfloat16, __nv_bfloat16>(c, stream);
  }
}

}  // namespace b200norm
