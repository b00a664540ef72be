// The tensor-core products, float16; the tiling rule and the status words.
#include "linear_mma_launch.cuh"

namespace b200norm {

template cudaError_t launch_mma_t<__half>(const Product&, const MmaPlan&, int, unsigned*,
                                          cudaStream_t);
extern template cudaError_t launch_mma_t<__nv_bfloat16>(const Product&, const MmaPlan&, int,
                                                        unsigned*, cudaStream_t);

extern template cudaError_t launch_mma_gated_t<__half>(const Product&, const MmaPlan&, int,
                                                       unsigned*, cudaStream_t);
extern template cudaError_t launch_mma_gated_t<__nv_bfloat16>(const Product&, const MmaPlan&, int,
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
static std::atomic<unsigned long long> g_linear_stall{0};

unsigned long long linear_stall_limit_ns() { return g_linear_stall.load(); }
void set_linear_stall(unsigned long long limit_ns) { g_linear_stall.store(limit_ns); }

static std::atomic<LinearWithhold> g_linear_withhold{LinearWithhold{0, 0}};

LinearWithhold linear_withhold() { return g_linear_withhold.load(); }
bool set_linear_withhold(unsigned site, unsigned limit_ns) {
  if (site != 0 && site != kSiteEmpty && site != kSiteDrained && site != kSiteResidual)
    return false;
  g_linear_withhold.store({site, limit_ns});
  return true;
}

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

// The tiling with the smallest estimated time.  The constants (microseconds) are
// fitted to 40 measured products from 128 x 768 x 768 to 4096^3 and meet most of
// them within a tenth: a slice of 64 of k takes 0.345 us in a pair's 256 x 256
// tile, 0.30 in a CTA's 128 x 128 and 0.36 in one of two 128 x 64 on an SM; a
// tile's end that nothing hides 0.8, a launch 3.0, and a sum split over a
// cluster 2.0 and 0.5 per part.  With a gate a tile has half as many of the result's N
// columns, and none is 128 x 64.
MmaPlan plan_mma(int64_t M, int64_t N, int64_t K, bool b_kc, bool gated, bool pieces, int sms) {
  const int64_t kblocks = (K + kMmaK - 1) / kMmaK;
  const int per = gated ? 2 : 1;
  const int64_t swapped = (N * per + kMmaRows - 1) / kMmaRows;
  // Few rows: the weight's rows fill the lanes.  (For 33 to 64 rows the ordinary
  // form is as fast unless there are few tiles to split K over: 64 x 16384 x 4096
  // 29.8 us against 35.2, but 64 x 4096 x 16384 31.8 against 32.8 without and
  // 45.2 against 33.9 with a residual, whose loads are not whole vectors here.)
  if (b_kc && M <= (swapped * 8 <= 2 * sms ? 64 : 32)) {
    MmaPlan p{1, M <= 16 ? 16 : M <= 32 ? 32 : 64, 1, true};
    while (p.splits < 8 && swapped * p.splits * 2 <= 2 * sms && kblocks / (p.splits * 2) >= 2)
      p.splits *= 2;
    return p;
  }
  MmaPlan best{1, gated || pieces ? 128 : 64, 1, false};
  double least = 0.0;
  const struct {
    int cg, bn, slots, most;
    double slice;
  } shapes[] = {{2, 256, sms / 2, 1, 0.345}, {1, 128, sms, 4, 0.30}, {1, 64, 2 * sms, 8, 0.36}};
  for (const auto& s : shapes) {
    if ((gated || pieces) && s.bn == 64) continue;
    for (int splits = 1; splits <= s.most && splits <= kblocks; splits *= 2) {
      const int64_t rows = s.cg * kMmaRows;
      const int64_t tiles = (M + rows - 1) / rows * ((N * per + s.bn - 1) / s.bn) * splits;
      const int64_t waves = (tiles + s.slots - 1) / s.slots;
      const int64_t slices = (kblocks + splits - 1) / splits;
      const double t = 3.0 + static_cast<double>(waves) *
                                 (static_cast<double>(slices) * s.slice + 0.8) +
                       (splits > 1 ? 2.0 + 0.5 * splits : 0.0);
      if (least == 0.0 || t < least) {
        least = t;
        best = {s.cg, s.bn, splits, false};
      }
    }
  }
  return best;
}

bool mma_plan_ok(const MmaPlan& p, int64_t M, int64_t K, bool a_kc, bool b_kc, bool gated) {
  const int64_t kblocks = (K + kMmaK - 1) / kMmaK;
  if (p.splits < 1 || p.splits > 8 || (p.splits & (p.splits - 1)) || p.splits > kblocks)
    return false;
  if (p.swap)
    return a_kc && b_kc && p.cg == 1 && M <= p.bn && (p.bn == 16 || p.bn == 32 || p.bn == 64);
  return (p.cg == 2 && p.bn == 256 && p.splits == 1) ||
         (p.cg == 1 && ((p.bn == 64 && !gated) || p.bn == 128));
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
  // in pieces a slice of K has three times the bytes (and six times the products); so counted, a
  // sum may be split into more parts than it has slices
  const int64_t K = p.piece_a ? 3 * ((p.K + kMmaK - 1) / kMmaK * kMmaK) : p.K;
  if (plan.cg == 0) plan = plan_mma(p.M, p.N, K, b_kc, p.gated, p.piece_a != 0, sms);
  else if (!mma_plan_ok(plan, p.M, K, a_kc, b_kc, p.gated)) return cudaErrorNotSupported;
  if (p.piece_a) return launch_mma_f32(p, plan, sms, status, stream);
  if (p.gated)
    return p.t == DType::F16 ? launch_mma_gated_t<__half>(p, plan, sms, status, stream)
                             : launch_mma_gated_t<__nv_bfloat16>(p, plan, sms, status, stream);
  return p.t == DType::F16 ? launch_mma_t<__half>(p, plan, sms, status, stream)
                           : launch_mma_t<__nv_bfloat16>(p, plan, sms, status, stream);
}

}  // namespace b200norm
