// linear_mma_launch.cuh -- host-side launch of the tensor-core products for one
// element type.
#pragma once

#include <atomic>

#include "linear_mma.cuh"

namespace b200norm {

// cuTensorMapEncodeTiled, looked up through the runtime (nullptr if missing).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn tensor_map_encoder();

// Boxes of `rows` rows by 64; what lies past an edge reads as zero and is not
// stored.  An operand: of `rows` by 64 of k (k contiguous), or squares of 64 by 64.
template <typename T>
bool encode_rows(CUtensorMap* map, const void* p, int64_t inner, int64_t outer, int64_t ld,
                 int rows) {
  EncodeFn fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * sizeof(T)};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)};
  const cuuint32_t one[2] = {1, 1};
  constexpr CUtensorMapDataType type = std::is_same<T, __half>::value
                                           ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
bool encode_operand(CUtensorMap* map, const Operand& o, int64_t n, int64_t k, int rows) {
  return o.k_contiguous ? encode_rows<T>(map, o.p, k, n, o.ld, rows)
                        : encode_rows<T>(map, o.p, n, k, o.ld, 64);
}

template <typename T, int CG, int BN, bool A_KC, bool B_KC, bool SWAP>
cudaError_t launch_mma_shape(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                             cudaStream_t stream) {
  using S = MmaShape<CG, BN, SWAP>;
  auto* fn = linear_mma_kernel<T, CG, BN, A_KC, B_KC, SWAP>;
  const Operand& a = SWAP ? p.b : p.a;
  const Operand& b = SWAP ? p.a : p.b;
  MmaArgs g;
  g.M = SWAP ? p.N : p.M;
  g.N = SWAP ? p.M : p.N;
  g.kblocks = static_cast<int>((p.K + kMmaK - 1) / kMmaK);
  g.tiles_m = static_cast<int>((g.M + CG * kMmaRows - 1) / (CG * kMmaRows));
  g.tiles_n = static_cast<int>((g.N + BN - 1) / BN);
  g.splits = plan.splits;
  g.e = p.epi;
  const void* outs[] = {p.epi.y, p.epi.z, p.epi.bias, p.epi.residual};
  g.vec = p.N % 8 == 0;
  for (const void* o : outs)
    if (reinterpret_cast<uintptr_t>(o) % 16 != 0) g.vec = false;
  g.status = status;
  // a wait lasts a tile at most: a second, and 4 us for each slice of K
  g.limit_ns = 1000000000ull + 4000ull * g.kblocks;
  g.stall = linear_stall_limit_ns() != 0;
  if (g.stall) g.limit_ns = linear_stall_limit_ns();
  const LinearWithhold withhold = linear_withhold();
  g.withhold = withhold.site;
  if (g.withhold) g.limit_ns = withhold.limit_ns * kMmaWithheld;
  CUtensorMap map_a, map_b;
  if (!encode_operand<T>(&map_a, a, g.M, p.K, kMmaRows) ||
      !encode_operand<T>(&map_b, b, g.N, p.K, S::kBRows))
    return cudaErrorInvalidValue;
  CUtensorMap map_y = {}, map_z = {}, map_r = {};
  if (!SWAP && g.vec && g.splits == 1) {  // results go by tensor copies
    const bool ok = encode_rows<T>(&map_y, p.epi.y, p.N, p.M, p.N, 32) &&
                    (!p.epi.z || encode_rows<T>(&map_z, p.epi.z, p.N, p.M, p.N, 32)) &&
                    (!p.epi.residual || encode_rows<T>(&map_r, p.epi.residual, p.N, p.M, p.N, 32));
    if (!ok) return cudaErrorInvalidValue;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // raise the dynamic shared-memory limit once per device (every time on
  // devices past the first 64)
  static std::atomic<unsigned long long> raised{0};
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(raised.load() & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(S::kSmem));
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit);
  }
  const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  const int cluster = CG == 2 ? 2 : g.splits;
  int64_t units = tiles;
  if (g.splits == 1) {  // persistent: as many as are resident at once
    const int64_t most = static_cast<int64_t>(sms) * (BN <= 64 ? 2 : 1) / CG;
    if (units > most) units = most;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  unsigned n = 0;
  if (cluster > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    n = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = add_pdl_attr(attr, n);
  return cudaLaunchKernelEx(&cfg, fn, map_a, map_b, map_y, map_z, map_r, g);
}

template <typename T, bool A_KC, bool B_KC>
cudaError_t launch_mma_layout(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                              cudaStream_t stream) {
  if constexpr (A_KC && B_KC) {
    if (plan.swap) {
      switch (plan.bn) {
        case 16: return launch_mma_shape<T, 1, 16, true, true, true>(p, plan, sms, status, stream);
        case 32: return launch_mma_shape<T, 1, 32, true, true, true>(p, plan, sms, status, stream);
        default: return launch_mma_shape<T, 1, 64, true, true, true>(p, plan, sms, status, stream);
      }
    }
  }
  if (plan.cg == 2)
    return launch_mma_shape<T, 2, 256, A_KC, B_KC, false>(p, plan, sms, status, stream);
  if (plan.bn == 128)
    return launch_mma_shape<T, 1, 128, A_KC, B_KC, false>(p, plan, sms, status, stream);
  return launch_mma_shape<T, 1, 64, A_KC, B_KC, false>(p, plan, sms, status, stream);
}

template <typename T>
cudaError_t launch_mma_t(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                         cudaStream_t stream) {
  if (p.a.k_contiguous && p.b.k_contiguous)
    return launch_mma_layout<T, true, true>(p, plan, sms, status, stream);
  if (p.a.k_contiguous)
    return launch_mma_layout<T, true, false>(p, plan, sms, status, stream);
  return launch_mma_layout<T, false, false>(p, plan, sms, status, stream);
}

}  // namespace b200norm
