// layer_launch.cuh -- host-side launch of the layer-normalization kernels for
// one (T, M) pair.
#pragma once

#include "launch_kernel.cuh"
#include "layer.cuh"
#include "layer.h"

namespace b200norm {

// Threads of a walking CTA: whole warps, no more than the row has vectors for.
inline int layer_walk_block(int64_t nvec) {
  const int64_t b = (nvec + 31) / 32 * 32;
  return static_cast<int>(b < kLayerThreads ? b : kLayerThreads);
}

// CTAs of the lane-group grid: six of 256 threads per SM.
constexpr int kLayerLaneCtas = 152 * 6;

constexpr int kLayerMaxCluster = 8;  // the portable cluster size

// Rows that are not whole vectors go by windows from these sizes on; smaller calls
// wait for one row's latency, and of short rows most of a warp is idle.  Element
// by element against windows, us: forward 1999 x 1027 float16 9.1, 10.2; 3001 x
// 1027 14.3, 13.6; 16384 x 1027 65.6, 48.4; gradient 304 x 1027 9.5, 10.2; 1999 x
// 1027 (without ds) 16.0, 12.7; 16384 x 1027 88.7, 53.2; 65536 x 67 84, 117; 65536 x
// 129 127, 118.
constexpr int kWindowHidden = 65, kWindowGradHidden = 128;
constexpr int64_t kWindowElements = 5 << 19, kWindowGradElements = 3 << 18;

// How a row is spread: `lane` threads of a warp, or `block` threads of each of
// `csize` CTAs, nv vectors per thread; nv 0: the row is walked.
struct LayerPlan {
  int lane, block, csize, nv;
};

inline LayerPlan plan_layer(int64_t rows, int64_t nvec) {
  LayerPlan p{0, 256, 1, 0};
  // at most two vectors per lane (with four, 16384 x 768 bf16 takes 22.6 us, 20.0 as
  // CTAs; 65536 x 512 float32 90, 80)
  if (nvec <= 64) {
    p.nv = nvec <= 32 ? 1 : 2;
    p.lane = 1;
    while (p.lane * p.nv < nvec) p.lane *= 2;
    return p;
  }
  // few rows: the latency of a row counts, so one vector per thread; many:
  // about 256 threads
  const int64_t want = rows <= 512 ? 512 : 256;
  int nv = 1;
  while (nv < 4 && nvec > want * nv) nv *= 2;
  while (nv < 8 && nvec > static_cast<int64_t>(kLayerThreads) * nv) nv *= 2;
  int c = 1;
  while (c < kLayerMaxCluster && nvec > static_cast<int64_t>(kLayerThreads) * nv * c) c *= 2;
  if (nvec > static_cast<int64_t>(kLayerThreads) * nv * c) return p;
  p.nv = nv;
  p.csize = c;
  p.block = static_cast<int>(((nvec + nv * c - 1) / (nv * c) + 31) / 32 * 32);
  return p;
}

template <typename T, typename M, int VE>
cudaError_t launch_layer_ve(const LayerCall& c, const LayerArgs<T, M>& a, cudaStream_t stream) {
  const int64_t nvec = c.hidden / VE;
  const LayerPlan p = plan_layer(c.rows, nvec);
  if (p.nv == 0 || c.rows * p.csize > 0x7fffffffLL)
    return launch_pdl(layer_walk_kernel<T, M, VE>, dim3(static_cast<unsigned>(c.rows)),
                      layer_walk_block(nvec), stream, a);
  using Fn = void (*)(const LayerArgs<T, M>, int, int);
  if (p.lane) {
    const Fn fn = p.nv == 1 ? layer_lane_kernel<T, M, VE, 1> : layer_lane_kernel<T, M, VE, 2>;
    const int64_t per = p.block / p.lane;
    int64_t grid = (c.rows + per - 1) / per;
    if (grid > kLayerLaneCtas) grid = kLayerLaneCtas;
    return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), p.block, stream, a, p.lane,
                      static_cast<int>(nvec));
  }
  const Fn fn = p.nv == 1   ? layer_cta_kernel<T, M, VE, 1>
                : p.nv == 2 ? layer_cta_kernel<T, M, VE, 2>
                : p.nv == 4 ? layer_cta_kernel<T, M, VE, 4>
                            : layer_cta_kernel<T, M, VE, 8>;
  return launch_clusters(fn, dim3(static_cast<unsigned>(c.rows * p.csize)), p.block, p.csize,
                         0, stream, a, p.block * p.csize, static_cast<int>(nvec));
}

// The CTAs of `fn` that the device holds at once; its shared-memory limit is
// raised and the driver is asked once per device, kernel and size.
template <class Fn>
cudaError_t layer_resident(Fn fn, int block, int smem, int* resident) {
  struct Key {
    int dev, block, smem;
    const void* fn;
  };
  static PlanCache<Key, int> cache;
  Key k;
  memset(&k, 0, sizeof(k));
  cudaError_t e = cudaGetDevice(&k.dev);
  if (e != cudaSuccess) return e;
  k.block = block;
  k.smem = smem;
  k.fn = reinterpret_cast<const void*>(fn);
  if (cache.get(k, resident)) return cudaSuccess;
  int sms = 0, per_sm = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, k.dev);
  if (e == cudaSuccess && smem > 0)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, block, smem);
  if (e != cudaSuccess) return e;
  *resident = (per_sm > 0 ? per_sm : 1) * sms;
  cache.put(k, *resident);
  return cudaSuccess;
}

inline bool on_vector(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The most vectors that a row's window has.
template <int VE>
int64_t window_vectors(int64_t hidden) {
  return (hidden + 2 * (VE - 1)) / VE;
}

// Rows that are not whole vectors, by windows; *done: whether their length allows it.
template <typename T, typename M, int VE>
cudaError_t launch_layer_window(const LayerCall& c, const LayerArgs<T, M>& a, cudaStream_t stream,
                                bool* done) {
  *done = false;
  const int64_t nvec = window_vectors<VE>(c.hidden);
  const int nv = nvec <= 256 ? 1 : VE == 4 && nvec > 512 ? 4 : 2;
  int csize = 1;
  while (csize < kLayerMaxCluster && nvec > static_cast<int64_t>(kLayerThreads) * nv * csize)
    csize *= 2;
  if (nvec > static_cast<int64_t>(kLayerThreads) * nv * csize) return cudaSuccess;
  const int block = static_cast<int>(((nvec + nv * csize - 1) / (nv * csize) + 31) / 32 * 32);
  constexpr int kMost = VE == 4 ? 4 : 2;
  auto* fn = nv == 1   ? layer_window_kernel<T, M, VE, 1>
             : nv == 2 ? layer_window_kernel<T, M, VE, 2>
                       : layer_window_kernel<T, M, VE, kMost>;
  int resident = 0;
  const int smem = nv * block * 16 * layer_window_pieces<T, M, VE>();
  cudaError_t e = layer_resident(fn, block, smem, &resident);
  if (e != cudaSuccess) return e;
  *done = true;
  const int parts = window_parts(c.rows, resident / csize, VE);
  return launch_clusters(fn, dim3(static_cast<unsigned>(parts * csize)), block, csize, smem,
                         stream, a, block * csize, parts);
}

template <typename T, typename M>
cudaError_t launch_layer_tm(const LayerCall& c, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  LayerArgs<T, M> a{static_cast<const T*>(c.x), static_cast<const T*>(c.skip),
                    static_cast<const M*>(c.gamma), static_cast<const M*>(c.beta),
                    static_cast<const T*>(c.bias), static_cast<T*>(c.y), static_cast<T*>(c.s),
                    c.mean, c.inv_std, c.rows, static_cast<int>(c.hidden),
                    1.0f / static_cast<float>(c.hidden), c.eps};
  if (c.vec) return launch_layer_ve<T, M, VE>(c, a, stream);
  if (c.hidden >= kWindowHidden && c.rows * c.hidden >= kWindowElements && on_vector(c.x) &&
      on_vector(c.skip) && on_vector(c.y) && on_vector(c.s)) {
    bool done;
    const cudaError_t e = launch_layer_window<T, M, VE>(c, a, stream, &done);
    if (done || e != cudaSuccess) return e;
  }
  return launch_layer_ve<T, M, 1>(c, a, stream);
}

// The streamed gradient: at most one wave of CTAs.  `apart`: rows of a part are a
// multiple of it apart.
template <typename T, typename M, class Fn>
cudaError_t launch_layer_grad_ring(Fn fn, LayerGradArgs<T, M>* a, int block, int csize,
                                   int tile_bytes, int tpr, int nvec, int slice,
                                   cudaStream_t stream, int apart = 1) {
  // CTAs of more than 256 threads fill an SM's registers alone; of the others
  // two share its memory
  const int budget = block > 256 ? 200 * 1024 : 100 * 1024;
  int stages = kLayerStages;
  while (stages > 2 && stages * tile_bytes > budget) --stages;
  const int smem = tile_bytes * stages;
  int resident = 0;
  const cudaError_t e = layer_resident(fn, block, smem, &resident);
  if (e != cudaSuccess) return e;
  const int fit = resident / csize > 1 ? resident / csize : 1;
  if (a->parts > fit) a->parts = fit;
  if (apart > 1) a->parts = window_parts(a->rows, a->parts, apart);
  unsigned* status = pipe_status_word();
  if (!status) return cudaErrorSymbolNotFound;
  int stall = 0;
  unsigned long long limit_ns = kLayerLimitNs;
  if (pipe_stalled()) {
    stall = kLayerNoCopies;
    limit_ns = pipe_stall_limit_ns();
  } else if (const unsigned long long ns = layer_withhold_limit_ns()) {
    stall = kLayerNoSums;
    limit_ns = ns;
  }
  return launch_clusters(fn, dim3(static_cast<unsigned>(a->parts * csize)), block, csize, smem,
                         stream, *a, tpr, nvec, slice, stages, status, limit_ns, stall);
}

// The one-pass gradient, NV vectors per thread of `block` threads of `csize` CTAs.
template <typename T, typename M, int VE, int NV, bool WINDOW = false>
cudaError_t launch_layer_grad_cta(const LayerGradCall& c, LayerGradArgs<T, M>* a, int csize,
                                  cudaStream_t stream) {
  const int nvec = static_cast<int>(WINDOW ? window_vectors<VE>(c.hidden) : c.hidden / VE);
  const int slice = (nvec + csize - 1) / csize;
  const int block = ((slice + NV - 1) / NV + 31) / 32 * 32;
  auto* fn = c.dbias ? layer_grad_ring_kernel<T, M, VE, NV, true, false, WINDOW>
                     : layer_grad_ring_kernel<T, M, VE, NV, false, false, WINDOW>;
  return launch_layer_grad_ring(fn, a, block, csize, 3 * layer_slot_bytes<T, VE>(slice), 0, nvec,
                                slice, stream, WINDOW ? VE : 1);
}

template <typename T, typename M, int VE, int NV>
cudaError_t launch_layer_grad_lane(const LayerGradCall& c, LayerGradArgs<T, M>* a,
                                   cudaStream_t stream) {
  const int nvec = static_cast<int>(c.hidden / VE);
  int tpr = 1;
  while (tpr * NV < nvec) tpr *= 2;
  const int per = kLayerGradLaneThreads / tpr;
  const int64_t blocks = (c.rows + per - 1) / per;
  if (a->parts > blocks) a->parts = static_cast<int>(blocks);
  auto* fn = c.dbias ? layer_grad_ring_kernel<T, M, VE, NV, true, true>
                     : layer_grad_ring_kernel<T, M, VE, NV, false, true>;
  return launch_layer_grad_ring(fn, a, kLayerGradLaneThreads, 1,
                                3 * layer_slot_bytes<T, VE>(per * nvec), tpr, nvec, nvec, stream);
}

// The gradient form that the row's length allows; sets a->parts to the parts
// that it writes.
template <typename T, typename M, int VE, bool WINDOW = false>
cudaError_t launch_layer_grad_ve(const LayerGradCall& c, LayerGradArgs<T, M>* a,
                                 cudaStream_t stream) {
  constexpr int kMost = layer_grad_most<VE>();
  a->ve = WINDOW ? 1 : VE;
  const int64_t nvec = WINDOW ? window_vectors<VE>(c.hidden) : c.hidden / VE;
  if constexpr (!WINDOW) {
    if (nvec <= 32) return launch_layer_grad_lane<T, M, VE, 1>(c, a, stream);
    if (nvec <= 64) return launch_layer_grad_lane<T, M, VE, 2>(c, a, stream);
  }
  // a CTA's slice of a row: what its threads hold, or (streamed) four stages of
  // three slices in 192 KB
  constexpr int64_t kSlice = VE == 8 ? 1024 : VE == 4 ? 1032 : kLayerThreads * kMost;
  int csize = 1;
  while (csize < kLayerMaxCluster && nvec > kSlice * csize) csize *= 2;
  if (nvec <= kSlice * csize) {
    // one vector per thread shortens a row, two let more rows be resident: 600 x 2048
    // bfloat16 8.0 us with one, 9.7 with two; 4096 x 1280 14.3, 17.1; 16384 x 1536
    // (without dbias) 43.3, 40.0; 4096 x 768 float32 14.3, 16.4
    const int64_t one = c.rows <= 1024 || VE == 4 ? 256 : 160;
    if (nvec <= one) return launch_layer_grad_cta<T, M, VE, 1, WINDOW>(c, a, csize, stream);
    if (kMost == 2 || nvec <= 512)
      return launch_layer_grad_cta<T, M, VE, 2, WINDOW>(c, a, csize, stream);
    return launch_layer_grad_cta<T, M, VE, kMost, WINDOW>(c, a, csize, stream);
  }
  if constexpr (WINDOW) return launch_layer_grad_ve<T, M, 1>(c, a, stream);
  a->ve = 1;
  cudaError_t e = launch_pdl(layer_grad_rows_kernel<T, M, VE>, dim3(static_cast<unsigned>(c.rows)),
                             layer_walk_block(nvec), stream, *a);
  if (e == cudaSuccess && (c.dgamma || c.dbeta || c.dbias))
    e = launch_pdl(layer_grad_cols_kernel<T, M>,
                   dim3(static_cast<unsigned>((c.hidden + 255) / 256), a->parts), 256, stream,
                   *a);
  return e;
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
                        layer_part_pitch(c.hidden), layer_grad_parts(c.rows, c.hidden), 1,
                        c.rows, static_cast<int>(c.hidden),
                        1.0f / static_cast<float>(c.hidden)};
  cudaError_t e = cudaSuccess;
  if (c.rows > 0) {
    if (c.vec)
      e = launch_layer_grad_ve<T, M, VE>(c, &a, stream);
    else if (c.hidden >= kWindowGradHidden && c.rows * c.hidden >= kWindowGradElements &&
             on_vector(c.dy) && on_vector(c.s) && on_vector(c.ds) && on_vector(c.dx))
      e = launch_layer_grad_ve<T, M, VE, true>(c, &a, stream);
    else
      e = launch_layer_grad_ve<T, M, 1>(c, &a, stream);
    if (e != cudaSuccess) return e;
  } else {
    a.parts = 0;  // empty sums
  }
  if (!c.dgamma && !c.dbeta && !c.dbias) return e;
  const auto blocks = [&](int cols) {
    return dim3(static_cast<unsigned>((c.hidden + cols - 1) / cols), 3);
  };
  if (c.hidden <= 2048)
    return launch_pdl(layer_grad_finish_kernel<T, M, 32>, blocks(32), kLayerFinishThreads<32>,
                      stream, a);
  return launch_pdl(layer_grad_finish_kernel<T, M, 128>, blocks(128), kLayerFinishThreads<128>,
                    stream, a);
}

}  // namespace b200norm
