// The linear operator without the tensor cores, float32.
#include "gated_few.cuh"
#include "linear_launch.cuh"

namespace b200norm {

__global__ void __launch_bounds__(256) linear_pieces_kernel(const PieceRows first,
                                                            const PieceRows second, int64_t n,
                                                            int64_t piece, bool vec, bool late) {
  if (!late) pdl_wait();
  pdl_trigger();
  const int64_t words = piece / 8;
  const int64_t total = (first.rows + second.rows) * words;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    int64_t row = i / words;
    const int64_t k = (i - row * words) * 8;
    const bool one = row < first.rows;
    if (!one) row -= first.rows;
    const float* p = (one ? first.src : second.src) + row * n + k;
    float f[8];
    if (vec && k + 8 <= n) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
      f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = k + e < n ? __ldcg(p + e) : 0.0f;
    }
    store_pieces<8>((one ? first.dst : second.dst) + row * 3 * piece + k, piece, f);
  }
  if (late) pdl_wait();
}

cudaError_t launch_pieces(const void* src0, void* dst0, int64_t rows0, const void* src1,
                          void* dst1, int64_t rows1, int64_t n, bool late, cudaStream_t stream) {
  const int64_t piece = piece_of(n);
  int64_t grid = ((rows0 + rows1) * (piece / 8) + 255) / 256;
  if (grid > 152 * 16) grid = 152 * 16;
  const PieceRows a{static_cast<const float*>(src0), static_cast<__nv_bfloat16*>(dst0), rows0};
  const PieceRows b{static_cast<const float*>(src1), static_cast<__nv_bfloat16*>(dst1), rows1};
  const bool vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(src0) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(src1) % 16 == 0;
  return launch_pdl(linear_pieces_kernel, dim3(static_cast<unsigned>(grid)), 256, stream, a, b, n,
                    piece, vec, late);
}

cudaError_t launch_plain_f32(const Product& p, cudaStream_t stream) {
  return launch_plain(p, stream);
}

template cudaError_t launch_rows<float>(const Product&, cudaStream_t);
template cudaError_t launch_dz<float>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_gated_dz<float>(const LinearDzCall&, cudaStream_t);
template cudaError_t launch_db<float>(const LinearDzCall&, bool, bool, cudaStream_t);
template cudaError_t launch_gated_few<float>(const GatedFewArgs&, void*, cudaStream_t);

}  // namespace b200norm
