// heads.h -- host-side interface between the C ABI and the kernels of the query
// and key heads: position rotation, with or without an RMS norm of each head.
#pragma once

#include "launch.h"

namespace b200norm {

constexpr int kMaxHeadSize = 1024;
constexpr int64_t kMaxHeads = int64_t{1} << 16;

// Element (b, t, h, d) of a tensor of heads at p[b * batch + t * token + h * head + d].
struct HeadStrides {
  int64_t batch, token, head;
};

// One tensor of heads (heads 0: absent).
struct HeadSet {
  const void* x;
  const void* dy;      // gradient only
  const void* gamma;   // null: ones
  void* y;             // the result (gradient: dx; null: not wanted)
  void* dgamma;        // gradient only (null: not wanted)
  int64_t heads;
  HeadStrides xs, dys, ys;
};

struct HeadsCall {
  HeadSet set[2];         // queries, keys
  const void* positions;  // int32 or int64
  bool pos64;
  int64_t pos_batch, pos_token;
  const double* inv_freq;  // rot / 2 radians per position
  int64_t batch, seq;
  int size, rot;
  bool interleaved, norm;
  bool inverse;            // forward only
  float scale, eps;
  DType t, m;
  float* part;             // gradient: sums over rows, head_parts() of them
};

// Lanes and steps of the row layout for a call (heads.cuh).
struct HeadsPlan {
  int ve;        // elements per access
  int units;     // pairs of accesses in a row
  int lanes;     // per row: a power of two, at most 32
  int sets;      // units a lane holds
};
HeadsPlan plan_heads(const HeadsCall& c, bool gradient);

// Parts of the sums behind dgamma, of queries and of keys: CTAs of each.
struct HeadParts {
  int q, k;
};
HeadParts head_parts(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t size);
inline size_t head_parts_bytes(HeadParts p, int64_t size) {
  return (static_cast<size_t>(p.q + p.k) * size * 4 + 255) / 256 * 256;
}

cudaError_t launch_heads(const HeadsCall& c, cudaStream_t stream);
cudaError_t launch_heads_grad(const HeadsCall& c, cudaStream_t stream);

}  // namespace b200norm
