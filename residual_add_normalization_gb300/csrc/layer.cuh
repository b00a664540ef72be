// layer.cuh -- layer normalization over the last axis, with the residual add
// fused in, and its gradients (sm_103a).
//
//   S = round_T((x + skip) + bias)            S = x without a skip
//   y = round_T((S - mu) * r * gamma + beta), mu = mean(S), r = 1/sqrt(var + eps)
//
// With u = (S - mu) * r, g = dy * gamma and n the row length:
//
//   dS     = r * (g - mean(g) - u * mean(g * u)) + ds
//   dgamma = sum over rows of dy * u,  dbeta = sum of dy,  dbias = sum of dS
//
// All of it is bound by HBM: about ten operations per element against 6 to 16
// bytes.  Statistics and sums are binary32; each stored value is rounded once
// (dbias sums dS before its rounding).
#pragma once

#include "common.cuh"

namespace b200norm {

template <typename T, typename M>
struct LayerArgs {
  const T* __restrict__ x;
  const T* __restrict__ skip;
  const M* __restrict__ gamma;
  const M* __restrict__ beta;
  const T* __restrict__ bias;
  T* __restrict__ y;
  T* __restrict__ s;
  float* __restrict__ mean;
  float* __restrict__ inv_std;
  int64_t rows;
  int n;
  float inv_n;
  float eps;
};

template <typename T, typename M>
struct LayerGradArgs {
  const T* __restrict__ dy;
  const T* __restrict__ s;
  const float* __restrict__ mean;
  const float* __restrict__ inv_std;
  const M* __restrict__ gamma;
  const T* __restrict__ ds;
  T* __restrict__ dx;
  M* __restrict__ dgamma;
  M* __restrict__ dbeta;
  T* __restrict__ dbias;
  float2* __restrict__ coef;    // per row: mean(g), mean(g * u)
  float* __restrict__ part;     // [parts][3][n]: dgamma, dbeta, dbias
  int parts;
  int64_t rows;
  int n;
  float inv_n;
};

constexpr int kLayerThreads = 512;

// VE parameters of type M as binary32 (one or two 16-byte loads, or scalars).
template <typename M, int VE>
__device__ __forceinline__ void ld_params(const M* p, float (&f)[VE]) {
  if constexpr (sizeof(M) * VE > 16) {
    constexpr int H = VE / 2;
    float a[H], b[H];
    unpack(ld_reuse<M, H>(p), a);
    unpack(ld_reuse<M, H>(p + H), b);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      f[i] = a[i];
      f[H + i] = b[i];
    }
  } else {
    unpack(ld_reuse<M, VE>(p), f);
  }
}

// S for one vector: binary32 sums in the stated order, one rounding to T.
template <typename T, typename M, int VE>
__device__ __forceinline__ Pack<T, VE> layer_sum(const LayerArgs<T, M>& a, int64_t off, int v) {
  const Pack<T, VE> x = ld_stream<T, VE>(a.x + off);
  if (!a.skip) return x;
  const Pack<T, VE> k = ld_stream<T, VE>(a.skip + off);
  float f[VE], kf[VE];
  unpack(x, f);
  unpack(k, kf);
#pragma unroll
  for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], kf[e]);
  if (a.bias) {
    float bf[VE];
    ld_params<T, VE>(a.bias + static_cast<int64_t>(v) * VE, bf);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], bf[e]);
  }
  return pack_from<T, VE>(f);
}

// Rows of any length: one CTA walks the row three times (sum, centred squares,
// output); the later walks are served by L2 for rows that fit there.  The mean
// is known before the squares are taken, so an offset costs no digits.
template <typename T, typename M, int VE>
__global__ void __launch_bounds__(kLayerThreads)
layer_walk_kernel(const LayerArgs<T, M> a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[33];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.n;
  const int nvec = a.n / VE;
  float sum = 0.0f;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const int64_t off = base + static_cast<int64_t>(v) * VE;
    const Pack<T, VE> s = layer_sum<T, M, VE>(a, off, v);
    float f[VE];
    unpack(s, f);
#pragma unroll
    for (int e = 0; e < VE; ++e) sum += f[e];
    if (a.s) st_stream<T, VE>(a.s + off, s);
  }
  const float mu = cta_sum(sum, red) * a.inv_n;
  float sq = 0.0f;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    float f[VE];
    unpack(layer_sum<T, M, VE>(a, base + static_cast<int64_t>(v) * VE, v), f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float d = f[e] - mu;
      sq = fmaf(d, d, sq);
    }
  }
  __syncthreads();  // red is read by every thread above
  const float r = rsqrtf(fmaf(cta_sum(sq, red), a.inv_n, a.eps));
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const int64_t off = base + static_cast<int64_t>(v) * VE;
    float f[VE], gf[VE];
    unpack(layer_sum<T, M, VE>(a, off, v), f);
    ld_params<M, VE>(a.gamma + static_cast<int64_t>(v) * VE, gf);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = (f[e] - mu) * r * gf[e];
    if (a.beta) {
      float bf[VE];
      ld_params<M, VE>(a.beta + static_cast<int64_t>(v) * VE, bf);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] += bf[e];
    }
    st_stream<T, VE>(a.y + off, pack_from<T, VE>(f));
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[blockIdx.x] = mu;
    if (a.inv_std) a.inv_std[blockIdx.x] = r;
  }
}

// dS of one vector from its operands (without ds).
template <int VE>
__device__ __forceinline__ void layer_dx(const float (&g)[VE], const float (&u)[VE], float r,
                                         float c1, float c2, float (&d)[VE]) {
#pragma unroll
  for (int e = 0; e < VE; ++e) d[e] = r * (g[e] - c1 - u[e] * c2);
}

// Gradient, rows of any length: one CTA per row takes the two row means, keeps
// them for the column kernel, and writes dS.
template <typename T, typename M, int VE>
__global__ void __launch_bounds__(kLayerThreads)
layer_grad_rows_kernel(const LayerGradArgs<T, M> a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 red[33];
  const int64_t row = blockIdx.x, base = row * a.n;
  const int nvec = a.n / VE;
  const float mu = a.mean[row], r = a.inv_std[row];
  float2 acc = make_float2(0.0f, 0.0f);
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const int64_t off = base + static_cast<int64_t>(v) * VE;
    float dy[VE], s[VE], gm[VE];
    unpack(ld_reuse<T, VE>(a.dy + off), dy);
    unpack(ld_reuse<T, VE>(a.s + off), s);
    ld_params<M, VE>(a.gamma + static_cast<int64_t>(v) * VE, gm);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float g = dy[e] * gm[e];
      acc.x += g;
      acc.y = fmaf(g, (s[e] - mu) * r, acc.y);
    }
  }
  acc = cta_sum2(acc, red);
  const float c1 = acc.x * a.inv_n, c2 = acc.y * a.inv_n;
  if (threadIdx.x == 0) a.coef[row] = make_float2(c1, c2);
  if (!a.dx) return;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const int64_t off = base + static_cast<int64_t>(v) * VE;
    float g[VE], u[VE], gm[VE], d[VE];
    unpack(ld_reuse<T, VE>(a.dy + off), g);
    unpack(ld_reuse<T, VE>(a.s + off), u);
    ld_params<M, VE>(a.gamma + static_cast<int64_t>(v) * VE, gm);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      g[e] *= gm[e];
      u[e] = (u[e] - mu) * r;
    }
    layer_dx<VE>(g, u, r, c1, c2, d);
    if (a.ds) {
      float h[VE];
      unpack(ld_stream<T, VE>(a.ds + off), h);
#pragma unroll
      for (int e = 0; e < VE; ++e) d[e] += h[e];
    }
    st_stream<T, VE>(a.dx + off, pack_from<T, VE>(d));
  }
}

// Column sums of the same: CTA (stripe, part) adds its part's rows, a column
// per thread, in row order.
template <typename T, typename M>
__global__ void __launch_bounds__(256)
layer_grad_cols_kernel(const LayerGradArgs<T, M> a) {
  pdl_wait();
  pdl_trigger();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= a.n) return;
  const int part = blockIdx.y;
  const int64_t r0 = a.rows * part / a.parts, r1 = a.rows * (part + 1) / a.parts;
  const float gm = to_f32(a.gamma[col]);
  float dg = 0.0f, db = 0.0f, dc = 0.0f;
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t off = row * a.n + col;
    const float dy = to_f32(a.dy[off]), r = a.inv_std[row];
    const float u = (to_f32(a.s[off]) - a.mean[row]) * r;
    dg = fmaf(dy, u, dg);
    db += dy;
    if (a.dbias) {
      const float2 c = a.coef[row];
      float d = r * (dy * gm - c.x - u * c.y);
      if (a.ds) d += to_f32(a.ds[off]);
      dc += d;
    }
  }
  float* p = a.part + static_cast<int64_t>(part) * 3 * a.n + col;
  p[0] = dg;
  p[a.n] = db;
  if (a.dbias) p[2 * static_cast<int64_t>(a.n)] = dc;
}

// The parts' sums added in a fixed order: a CTA takes 32 columns of one of the
// three outputs, its 32 warps every 32nd part, then the warps' sums are added
// through shared memory.
template <typename T, typename M>
__global__ void __launch_bounds__(1024)
layer_grad_finish_kernel(const LayerGradArgs<T, M> a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const int which = blockIdx.y;
  if (which == 0 ? !a.dgamma : which == 1 ? !a.dbeta : !a.dbias) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (col < a.n)
    for (int p = warp; p < a.parts; p += 32)
      t += a.part[(static_cast<int64_t>(p) * 3 + which) * a.n + col];
  red[warp][lane] = t;
  __syncthreads();
  // warp w now adds column w over the 32 warps
  t = warp_sum(red[lane][warp]);
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && out < a.n) {
    if (which == 0) a.dgamma[out] = from_f32<M>(t);
    else if (which == 1) a.dbeta[out] = from_f32<M>(t);
    else a.dbias[out] = from_f32<T>(t);
  }
}

}  // namespace b200norm
