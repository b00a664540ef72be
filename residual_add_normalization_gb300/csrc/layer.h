// layer.h -- host-side interface between the C ABI and the layer-normalization
// kernels (layer.cuh).  Each function enqueues on `stream` and returns the CUDA
// error of the launch.
#pragma once

#include "launch.h"

namespace b200norm {

struct LayerCall {
  const void* x;
  const void* skip;   // null: S = x
  const void* gamma;
  const void* beta;   // null: none
  const void* bias;   // null: none
  void* y;
  void* s;            // null: not stored
  float* mean;        // null: not stored
  float* inv_std;     // null: not stored
  int64_t rows;
  int64_t hidden;
  DType t, m;
  float eps;
  bool vec;           // every row and pointer is whole 16-byte vectors
};

struct LayerGradCall {
  const void* dy;
  const void* s;
  const float* mean;
  const float* inv_std;
  const void* gamma;
  const void* ds;     // null: nothing arrives through S
  void* dx;           // null: not wanted (as the three below)
  void* dgamma;
  void* dbeta;
  void* dbias;
  int64_t rows;
  int64_t hidden;
  DType t, m;
  void* workspace;    // layer_grad_workspace_bytes(rows, hidden)
  bool vec;
};

// Partial column sums a gradient call keeps: one set of (dgamma, dbeta, dbias)
// rows per part, later added in part order (no atomics, so equal calls give
// equal bits).  At most six parts per SM (CTAs of short rows; 16384 x 1024
// bfloat16 takes 33 us with four per SM, 47 with two), fewer for long rows, and
// two rows in each once every SM has one (608 x 1024: 7.2 us, 8.5 with one row).
constexpr int kLayerMaxParts = 912;
inline int64_t layer_part_pitch(int64_t hidden) { return (hidden + 3) / 4 * 4; }
inline int layer_grad_parts(int64_t rows, int64_t hidden) {
  int64_t p = rows > 152 ? (rows / 2 > 152 ? rows / 2 : 152) : rows;
  const int64_t most = (int64_t{1} << 24) / hidden;
  if (p > most) p = most;
  if (p > kLayerMaxParts) p = kLayerMaxParts;
  return static_cast<int>(p < 1 ? 1 : p);
}
inline size_t layer_grad_workspace_bytes(int64_t rows, int64_t hidden) {
  const size_t stats = (static_cast<size_t>(rows) * 8 + 255) / 256 * 256;
  return stats + static_cast<size_t>(layer_grad_parts(rows, hidden)) * 3 * layer_part_pitch(hidden) * 4;
}

// `parts` CTAs (clusters) of which each takes every parts-th of `rows` rows, if
// rows of one part must be a multiple of `ve` apart: one row each, or a multiple of
// `ve` of them, never more than there are rows (the workspace has no more parts).
inline int window_parts(int64_t rows, int64_t parts, int ve) {
  if (parts >= rows || rows <= ve) return static_cast<int>(rows);
  return static_cast<int>(parts > ve ? parts - parts % ve : ve);
}

// A test's limit for the waits of launches whose CTAs do not send one another their
// sums of a long row (0: normal ones).
unsigned long long layer_withhold_limit_ns();
void set_layer_withhold(unsigned long long limit_ns);

cudaError_t launch_layer(const LayerCall& c, cudaStream_t stream);
cudaError_t launch_layer_grad(const LayerGradCall& c, cudaStream_t stream);

// One (T, M) pair each, in its own translation unit.
template <typename T, typename M>
cudaError_t launch_layer_tm(const LayerCall& c, cudaStream_t stream);
template <typename T, typename M>
cudaError_t launch_layer_grad_tm(const LayerGradCall& c, cudaStream_t stream);

}  // namespace b200norm
