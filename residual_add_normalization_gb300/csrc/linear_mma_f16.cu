// The tensor-core products, float16; the tiling rule and the status words.
#include "linear_mma_launch.cuh"

namespace b200norm {

template cudaError_t launch_mma_t<__half>(const Product&, const MmaPlan&, int, unsigned*,
                                          cudaStream_t);
extern template cudaError_t launch_mma_t<__nv_bfloat16>(const Product&, const MmaPlan&, int,
                                                        unsigned*, cudaStream_t);

EncodeFn tensor_map_encoder() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn fn = cached.load();
  if (fn) return fn;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  fn = reinterpret_cast<EncodeFn>(p);
  cached.store(fn);
  return fn;
}

__device__ unsigned g_linear_status[2];

unsigned* linear_status_words() {
  constexpr int kCachedDevices = 64;  // devices past these are looked up every time
  static std::atomic<unsigned*> cache[kCachedDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
    cudaGetLastError();
    return nullptr;
  }
  unsigned* p = dev < kCachedDevices ? cache[dev].load() : nullptr;
  if (p) return p;
  void* addr = nullptr;
  if (cudaGetSymbolAddress(&addr, g_linear_status) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  p = static_cast<unsigned*>(addr);
  if (dev < kCachedDevices) cache[dev].store(p);
  return p;
}

MmaPlan plan_mma(int64_t M, int64_t N, int64_t K, bool b_kc, int sms) {
  const int64_t kblocks = (K + kMmaK - 1) / kMmaK;
  MmaPlan p{1, 64, 1, false};
  if (b_kc && M <= 64) {
    p.swap = true;
    p.bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const int64_t tiles = (N + kMmaRows - 1) / kMmaRows;
    while (p.splits < 8 && tiles * p.splits * 2 <= 2 * sms && kblocks / (p.splits * 2) >= 4)
      p.splits *= 2;
    return p;
  }
  // Estimated cycles: waves of tiles x (slices of K x cycles per slice + a
  // tile's start and end).
  double best = 0.0;
  const struct { int cg, bn; double slice; } shapes[] = {{2, 256, 512.0}, {1, 128, 400.0}, {1, 64, 300.0}};
  for (const auto& s : shapes)
    for (int splits = 1; splits <= (s.cg == 2 ? 1 : 8); splits *= 2) {
      if (splits > 1 && kblocks / splits < 4) break;
      const int64_t rows = s.cg * kMmaRows;
      const int64_t tiles = (M + rows - 1) / rows * ((N + s.bn - 1) / s.bn) * splits;
      const int64_t slots = sms / s.cg;
      const int64_t waves = (tiles + slots - 1) / slots;
      const double t = static_cast<double>(waves) *
                       (static_cast<double>((kblocks + splits - 1) / splits) * s.slice + 1500.0 +
                        (splits > 1 ? 1500.0 : 0.0));
      if (best == 0.0 || t < best) {
        best = t;
        p = {s.cg, s.bn, splits, false};
      }
    }
  return p;
}

bool mma_plan_ok(const MmaPlan& p, int64_t M, int64_t K, bool a_kc, bool b_kc) {
  const int64_t kblocks = (K + kMmaK - 1) / kMmaK;
  if (p.splits < 1 || p.splits > 8 || (p.splits & (p.splits - 1)) || p.splits > kblocks)
    return false;
  if (p.swap)
    return a_kc && b_kc && p.cg == 1 && M <= p.bn && (p.bn == 16 || p.bn == 32 || p.bn == 64);
  return (p.cg == 2 && p.bn == 256 && p.splits == 1) ||
         (p.cg == 1 && (p.bn == 64 || p.bn == 128));
}

cudaError_t launch_mma(const Product& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  unsigned* status = linear_status_words();
  if (!status) return cudaErrorSymbolNotFound;
  const bool a_kc = p.a.k_contiguous, b_kc = p.b.k_contiguous;
  MmaPlan plan = p.forced;
  if (plan.cg == 0) plan = plan_mma(p.M, p.N, p.K, b_kc, sms);
  else if (!mma_plan_ok(plan, p.M, p.K, a_kc, b_kc)) return cudaErrorNotSupported;
  return p.t == DType::F16 ? launch_mma_t<__half>(p, plan, sms, status, stream)
                           : launch_mma_t<__nv_bfloat16>(p, plan, sms, status, stream);
}

}  // namespace b200norm
