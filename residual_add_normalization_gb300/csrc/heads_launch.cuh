// heads_launch.cuh -- host-side launch of the head kernels for one element type.
#pragma once

#include <atomic>

#include "heads.cuh"
#include "launch_kernel.cuh"

namespace b200norm {

inline HeadsArgs head_args(const HeadsCall& c, const HeadsPlan& p) {
  HeadsArgs g = {};
  g.c = c;
  g.tokens = static_cast<unsigned>(c.batch * c.seq);
  g.seq = static_cast<unsigned>(c.seq);
  g.units = p.units;
  g.lanes = p.lanes;
  g.full = c.rot == c.size;
  g.whole = p.ve < 4 || c.rot / 2 % (p.ve / 2) == 0;  // (half layout: of whole accesses)
  const int rows = 32 / p.lanes;
  for (int n = 0; n < 2; ++n)
    g.steps[n] = static_cast<int>((c.set[n].heads + rows - 1) / rows);
  return g;
}

template <int N>
using Num = std::integral_constant<int, N>;

// f(VE, K, LANES, FORM) for the row layout: K is rounded up to what has a kernel; LANES and
// FORM are 0 (known at run time) but for the usual rows of whole 16-byte vectors.
template <typename T, class F>
cudaError_t with_head_layout(const HeadsCall& c, const HeadsPlan& p, F&& f) {
  constexpr int kVec = 16 / sizeof(T);
  const int form = c.rot != c.size ? 0 : c.interleaved ? 2 : 1;
  if (p.ve == kVec) {
    if (p.sets <= 1) {
      auto lanes = [&](auto n) {
        if (form == 1) return f(Num<kVec>(), Num<1>(), n, Num<1>());
        if (form == 2) return f(Num<kVec>(), Num<1>(), n, Num<2>());
        return f(Num<kVec>(), Num<1>(), n, Num<0>());
      };
      if (p.lanes == 4) return lanes(Num<4>());
      if (p.lanes == 8) return lanes(Num<8>());
      if (p.lanes == 16) return lanes(Num<16>());
      return f(Num<kVec>(), Num<1>(), Num<0>(), Num<0>());
    }
    if (p.sets <= 2) return f(Num<kVec>(), Num<2>(), Num<0>(), Num<0>());
    if constexpr (sizeof(T) == 4) return f(Num<kVec>(), Num<4>(), Num<0>(), Num<0>());
  }
  if constexpr (sizeof(T) == 2) {
    if (p.ve == 4) {
      if (p.sets <= 1) return f(Num<4>(), Num<1>(), Num<0>(), Num<0>());
      return f(Num<4>(), Num<2>(), Num<0>(), Num<0>());
    }
    if (p.ve == 2) {
      if (p.sets <= 1) return f(Num<2>(), Num<1>(), Num<0>(), Num<0>());
      if (p.sets <= 2) return f(Num<2>(), Num<2>(), Num<0>(), Num<0>());
      if (p.sets <= 4) return f(Num<2>(), Num<4>(), Num<0>(), Num<0>());
      return f(Num<2>(), Num<8>(), Num<0>(), Num<0>());
    }
  }
  if (p.sets <= 1) return f(Num<1>(), Num<1>(), Num<0>(), Num<0>());
  if (p.sets <= 2) return f(Num<1>(), Num<2>(), Num<0>(), Num<0>());
  if (p.sets <= 4) return f(Num<1>(), Num<4>(), Num<0>(), Num<0>());
  return f(Num<1>(), Num<16>(), Num<0>(), Num<0>());
}

// Raises a kernel's dynamic shared-memory limit once per device (every time on devices
// past the first 64).
template <class Fn>
cudaError_t head_raise(Fn fn, size_t smem, std::atomic<unsigned long long>& raised) {
  if (smem <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (raised.load() & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess) raised.fetch_or(bit);
  return e;
}

// CTAs of a kernel that are resident at once (152 if unknown); `seen` keeps the last answer,
// which depends on the device and on the shared memory.
template <class Fn>
int64_t head_resident(Fn fn, size_t smem, std::atomic<unsigned long long>& seen) {
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  const unsigned long long key = (static_cast<unsigned long long>(dev) << 32 | smem) + 1;
  const unsigned long long last = seen.load();  // key << 16 | CTAs
  if (last >> 16 == key) return static_cast<int64_t>(last & 0xffff);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, 32 * kHeadWarps, smem) !=
          cudaSuccess)
    return 152;
  const int64_t ctas = static_cast<int64_t>(sms) * per;
  if (ctas <= 0xffff) seen.store(key << 16 | static_cast<unsigned long long>(ctas));
  return ctas;
}

template <typename T>
cudaError_t launch_heads_t(const HeadsCall& c, cudaStream_t stream) {
  const HeadsPlan p = plan_heads(c, false);
  HeadsArgs g = head_args(c, p);
  const int64_t all = (static_cast<int64_t>(g.steps[0]) + g.steps[1]) * g.tokens;
  return with_head_layout<T>(c, p, [&](auto ve, auto k, auto lanes, auto form) {
    constexpr int VE = decltype(ve)::value, K = decltype(k)::value, L = decltype(lanes)::value;
    auto go = [&](auto norm) {
      auto* fn = heads_kernel<T, VE, K, L, decltype(form)::value, decltype(norm)::value>;
      static std::atomic<unsigned long long> raised{0}, seen{0};
      g.pitch = p.lanes * K * VE;
      const size_t smem = head_smem<T, VE, K>(g, false);
      if (const cudaError_t e = head_raise(fn, smem, raised)) return e;
      int64_t grid = (all + kHeadWarps - 1) / kHeadWarps;
      // resident at once: a warp's share is an equal part of all steps
      const int64_t most = grid > 1 ? head_resident(fn, smem, seen) : 1;
      if (grid > most) grid = most;
      return launch_clusters(fn, dim3(static_cast<unsigned>(grid)), 32 * kHeadWarps, 1, smem,
                             stream, g);
    };
    return c.norm ? go(std::true_type()) : go(std::false_type());
  });
}

template <typename T>
cudaError_t launch_heads_grad_t(const HeadsCall& c, cudaStream_t stream) {
  const HeadsPlan p = plan_heads(c, true);
  HeadsArgs g = head_args(c, p);
  const HeadParts parts = head_parts(g.tokens, c.set[0].heads, c.set[1].heads, c.size);
  g.parts[0] = parts.q;
  g.parts[1] = parts.k;
  return with_head_layout<T>(c, p, [&](auto ve, auto k, auto lanes, auto form) {
    constexpr int VE = decltype(ve)::value, K = decltype(k)::value, L = decltype(lanes)::value;
    static std::atomic<unsigned long long> raised{0};
    g.pitch = p.lanes * K * VE;
    auto* fn = heads_grad_kernel<T, VE, K, L, decltype(form)::value>;
    const size_t smem = head_smem<T, VE, K>(g, true);
    if (const cudaError_t e = head_raise(fn, smem, raised)) return e;
    return launch_clusters(fn, dim3(static_cast<unsigned>(parts.q + parts.k)), 32 * kHeadWarps, 1,
                           smem, stream, g);
  });
}

// dgamma of both tensors from `parts`, of type M.
template <typename M>
cudaError_t launch_heads_dgamma_t(const HeadsCall& c, HeadParts parts, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((c.size + 31) / 32), 2);
  return launch_pdl(heads_dgamma_kernel<M>, grid, 1024, stream, static_cast<const float*>(c.part),
                    static_cast<M*>(c.set[0].dgamma), static_cast<M*>(c.set[1].dgamma), c.size,
                    parts.q, parts.k);
}

}  // namespace b200norm
