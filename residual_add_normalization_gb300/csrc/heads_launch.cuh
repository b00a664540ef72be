// heads_launch.cuh -- host-side launch of the head kernels for one element type.
#pragma once

#include "heads.cuh"
#include "launch_kernel.cuh"

namespace b200norm {

// Warps that a forward call spreads a token's heads over while the GPU has room.
constexpr int64_t kHeadFill = 152 * 16;

inline HeadsArgs head_args(const HeadsCall& c, const HeadsPlan& p) {
  HeadsArgs g = {};
  g.c = c;
  g.tokens = static_cast<unsigned>(c.batch * c.seq);
  g.seq = static_cast<unsigned>(c.seq);
  g.units = p.units;
  g.lanes = p.lanes;
  const int rows = 32 / p.lanes;
  for (int n = 0; n < 2; ++n)
    g.steps[n] = static_cast<int>((c.set[n].heads + rows - 1) / rows);
  return g;
}

// f(VE, K) for the row layout: K is rounded up to what has a kernel.
template <typename T, class F>
cudaError_t with_head_layout(const HeadsPlan& p, F&& f) {
  constexpr int kVec = 16 / sizeof(T);
  if (p.ve == kVec) {
    if (p.sets <= 1) return f(std::integral_constant<int, kVec>(), std::integral_constant<int, 1>());
    if (p.sets <= 2) return f(std::integral_constant<int, kVec>(), std::integral_constant<int, 2>());
    if constexpr (sizeof(T) == 4)
      return f(std::integral_constant<int, kVec>(), std::integral_constant<int, 4>());
  }
  if constexpr (sizeof(T) == 2) {
    if (p.ve == 2) {
      if (p.sets <= 2) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 2>());
      return f(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
    }
  }
  if (p.sets <= 4) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 1>(), std::integral_constant<int, 16>());
}

template <typename T>
cudaError_t launch_heads_t(const HeadsCall& c, cudaStream_t stream) {
  const HeadsPlan p = plan_heads(c, false);
  HeadsArgs g = head_args(c, p);
  const int64_t all = static_cast<int64_t>(g.steps[0]) + g.steps[1];
  int64_t splits = (kHeadFill + g.tokens - 1) / g.tokens;
  if (splits > all) splits = all;
  g.splits = static_cast<int>(splits);
  const int64_t items = splits * g.tokens;
  const dim3 grid(static_cast<unsigned>((items + kHeadWarps - 1) / kHeadWarps));
  return with_head_layout<T>(p, [&](auto ve, auto k) {
    constexpr int VE = decltype(ve)::value, K = decltype(k)::value;
    return c.norm ? launch_pdl(heads_kernel<T, VE, K, true>, grid, 32 * kHeadWarps, stream, g)
                  : launch_pdl(heads_kernel<T, VE, K, false>, grid, 32 * kHeadWarps, stream, g);
  });
}

template <typename T>
cudaError_t launch_heads_grad_t(const HeadsCall& c, cudaStream_t stream) {
  const HeadsPlan p = plan_heads(c, true);
  HeadsArgs g = head_args(c, p);
  const HeadParts parts = head_parts(g.tokens, c.set[0].heads, c.set[1].heads);
  g.parts[0] = parts.q;
  g.parts[1] = parts.k;
  // a part's warps take tokens, or parts of a token's heads where there are more warps
  const int most = g.steps[0] > g.steps[1] ? g.steps[0] : g.steps[1];
  const int64_t warps = static_cast<int64_t>(parts.q + parts.k) * kHeadWarps;
  int64_t splits = warps / (2 * static_cast<int64_t>(g.tokens));
  if (splits > most) splits = most;
  g.splits = static_cast<int>(splits < 1 ? 1 : splits);
  const dim3 grid(static_cast<unsigned>(parts.q + parts.k));
  cudaError_t e = with_head_layout<T>(p, [&](auto ve, auto k) {
    return launch_pdl(heads_grad_kernel<T, decltype(ve)::value, decltype(k)::value>, grid,
                      32 * kHeadWarps, stream, g);
  });
  return e;
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
