// The head kernels' host side: row layout, parts, and the element type's launch.
#include "heads_launch.cuh"

namespace b200norm {

extern template cudaError_t launch_heads_t<float>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_t<__half>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_t<__nv_bfloat16>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_grad_t<float>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_grad_t<__half>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_grad_t<__nv_bfloat16>(const HeadsCall&, cudaStream_t);
extern template cudaError_t launch_heads_dgamma_t<float>(const HeadsCall&, HeadParts,
                                                         cudaStream_t);
extern template cudaError_t launch_heads_dgamma_t<__half>(const HeadsCall&, HeadParts,
                                                          cudaStream_t);
extern template cudaError_t launch_heads_dgamma_t<__nv_bfloat16>(const HeadsCall&, HeadParts,
                                                                 cudaStream_t);

namespace {

// Whether accesses of n elements fit a tensor: its start, and the steps that are taken.
bool fits(const HeadsCall& c, const HeadSet& s, const void* p, const HeadStrides& st, int n,
          size_t es) {
  if (!p || s.heads == 0) return true;
  return reinterpret_cast<uintptr_t>(p) % (n * es) == 0 && (c.batch == 1 || st.batch % n == 0) &&
         (c.seq == 1 || st.token % n == 0) && (s.heads == 1 || st.head % n == 0);
}

}  // namespace

HeadsPlan plan_heads(const HeadsCall& c, bool gradient) {
  const size_t es = dtype_size(c.t);
  HeadsPlan p = {};
  const int whole = static_cast<int>(16 / es);
  // (accesses of 8 bytes: rows of 16-bit types of which a lane holds two units at most)
  for (p.ve = whole; p.ve > 1; p.ve = es == 4 ? 1 : p.ve / 2) {
    bool ok = c.size % p.ve == 0 && (c.interleaved || c.rot / 2 % p.ve == 0) &&
              (p.ve == whole || p.ve != 4 || c.size <= 32 * 2 * 2 * p.ve);
    for (const HeadSet& s : c.set)
      ok = ok && fits(c, s, s.x, s.xs, p.ve, es) && fits(c, s, s.y, s.ys, p.ve, es) &&
           (!gradient || fits(c, s, s.dy, s.dys, p.ve, es));
    if (ok) break;
  }
  const int vectors = (c.size + p.ve - 1) / p.ve;
  p.units = (vectors + 1) / 2;
  p.lanes = 1;
  // The fewest lanes that hold a row in so many units each (more rows a step; with one unit a
  // lane 4096 x 20 x 33 bf16 took 20.0 us with the norm, 11.7 with four, gradients 49 and 22;
  // 100 elements, four at a time, 18.3 and 16.2, 35 and 27).  Whole 16-byte accesses: one.
  const int most = p.ve == whole ? 1 : p.ve == 1 ? 4 : p.ve == 2 && !gradient ? 4 : 2;
  while (p.lanes < 32 && p.lanes * most < p.units) p.lanes *= 2;
  p.sets = (p.units + p.lanes - 1) / p.lanes;
  return p;
}

HeadParts head_parts(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t size) {
  // CTAs in proportion to the steps that the tensors' rows take (of a 16-bit type's whole
  // accesses; other layouts are balanced less well), two for each of 152 SMs while a warp
  // has two steps
  int64_t rows = 32;
  while (rows > 1 && rows * size > 32 * 16) rows /= 2;
  const int64_t q = (q_heads + rows - 1) / rows, k = (k_heads + rows - 1) / rows;
  int64_t all = 152 * 2;
  const int64_t most = (tokens * (q + k) + 2 * kHeadWarps - 1) / (2 * kHeadWarps);
  if (all > most) all = most;
  if (all < 2) all = 2;
  if (k_heads == 0) return {static_cast<int>(all), 0};
  if (q_heads == 0) return {0, static_cast<int>(all)};
  int64_t part = (all * q + (q + k) / 2) / (q + k);
  part = part < 1 ? 1 : part > all - 1 ? all - 1 : part;
  return {static_cast<int>(part), static_cast<int>(all - part)};
}

cudaError_t launch_heads(const HeadsCall& c, cudaStream_t stream) {
  switch (c.t) {
    case DType::F32: return launch_heads_t<float>(c, stream);
    case DType::F16: return launch_heads_t<__half>(c, stream);
    default: return launch_heads_t<__nv_bfloat16>(c, stream);
  }
}

cudaError_t launch_heads_grad(const HeadsCall& c, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  HeadParts parts = {0, 0};
  if (c.batch * c.seq > 0) {
    parts = head_parts(c.batch * c.seq, c.set[0].heads, c.set[1].heads, c.size);
    switch (c.t) {
      case DType::F32: e = launch_heads_grad_t<float>(c, stream); break;
      case DType::F16: e = launch_heads_grad_t<__half>(c, stream); break;
      default: e = launch_heads_grad_t<__nv_bfloat16>(c, stream);
    }
  }
  if (e != cudaSuccess || (!c.set[0].dgamma && !c.set[1].dgamma)) return e;
  switch (c.m) {
    case DType::F32: return launch_heads_dgamma_t<float>(c, parts, stream);
    case DType::F16: return launch_heads_dgamma_t<__half>(c, parts, stream);
    default: return launch_heads_dgamma_t<__nv_bfloat16>(c, parts, stream);
  }
}

}  // namespace b200norm
