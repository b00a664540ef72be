// layer_launch.cuh -- host-side launch of the layer-normalization kernels for
// one (T, M) pair.
#pragma once

#include "layer.cuh"
#include "layer.h"

namespace b200norm {

template <class Fn, class... A>
cudaError_t launch_pdl(Fn fn, dim3 grid, int block, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = add_pdl_attr(attr, 0);
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Threads of a walking CTA: whole warps, no more than the row has vectors for.
inline int layer_walk_block(int64_t nvec) {
  const int64_t b = (nvec + 31) / 32 * 32;
  return static_cast<int>(b < kLayerThreads ? b : kLayerThreads);
}

template <typename T, typename M>
cudaError_t launch_layer_tm(const LayerCall& c, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  LayerArgs<T, M> a{static_cast<const T*>(c.x), static_cast<const T*>(c.skip),
                    static_cast<const M*>(c.gamma), static_cast<const M*>(c.beta),
                    static_cast<const T*>(c.bias), static_cast<T*>(c.y), static_cast<T*>(c.s),
                    c.mean, c.inv_std, c.rows, static_cast<int>(c.hidden),
                    1.0f / static_cast<float>(c.hidden), c.eps};
  const dim3 grid(static_cast<unsigned>(c.rows));
  if (c.vec)
    return launch_pdl(layer_walk_kernel<T, M, VE>, grid, layer_walk_block(c.hidden / VE), stream,
                      a);
  return launch_pdl(layer_walk_kernel<T, M, 1>, grid, layer_walk_block(c.hidden), stream, a);
}

template <typename T, typename M>
cudaError_t launch_layer_grad_tm(const LayerGradCall& c, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  const size_t stats = (static_cast<size_t>(c.rows) * 8 + 255) / 256 * 256;
  LayerGradArgs<T, M> a{static_cast<const T*>(c.dy), static_cast<const T*>(c.s), c.mean,
                        c.inv_std, static_cast<const M*>(c.gamma), static_cast<const T*>(c.ds),
                        static_cast<T*>(c.dx), static_cast<M*>(c.dgamma),
                        static_cast<M*>(c.dbeta), static_cast<T*>(c.dbias),
                        static_cast<float2*>(c.workspace),
                        reinterpret_cast<float*>(static_cast<char*>(c.workspace) + stats),
                        layer_grad_parts(c.rows, c.hidden), c.rows, static_cast<int>(c.hidden),
                        1.0f / static_cast<float>(c.hidden)};
  cudaError_t e = cudaSuccess;
  if (c.rows > 0) {
    const dim3 grid(static_cast<unsigned>(c.rows));
    e = c.vec ? launch_pdl(layer_grad_rows_kernel<T, M, VE>, grid,
                           layer_walk_block(c.hidden / VE), stream, a)
              : launch_pdl(layer_grad_rows_kernel<T, M, 1>, grid, layer_walk_block(c.hidden),
                           stream, a);
    if (e != cudaSuccess) return e;
    if (c.dgamma || c.dbeta || c.dbias)
      e = launch_pdl(layer_grad_cols_kernel<T, M>,
                     dim3(static_cast<unsigned>((c.hidden + 255) / 256), a.parts), 256, stream, a);
    if (e != cudaSuccess) return e;
  } else {
    a.parts = 0;  // empty sums
  }
  if (c.dgamma || c.dbeta || c.dbias)
    e = launch_pdl(layer_grad_finish_kernel<T, M>,
                   dim3(static_cast<unsigned>((c.hidden + 31) / 32), 3), 1024, stream, a);
  return e;
}

}  // namespace b200norm
