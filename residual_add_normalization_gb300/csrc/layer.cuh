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

#include "bulk.cuh"
#include "common.cuh"
#include "pair.cuh"

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
  float* __restrict__ part;     // [parts][3][pitch]: dgamma, dbeta, dbias, at part_at()
  int64_t pitch;                // n rounded up to four
  int parts;
  int ve;                       // elements per vector of the kernel that fills part
  int64_t rows;
  int n;
  float inv_n;
};

constexpr int kLayerThreads = 512;

// Where column `col` lies in a row of `part`: vectors of eight are kept as two
// planes of four, so that a warp's 16-byte stores are contiguous.
__device__ __forceinline__ int64_t part_at(int col, int n, int ve) {
  if (ve != 8) return col;
  return (static_cast<int64_t>((col >> 2) & 1) * (n >> 3) + (col >> 3)) * 4 + (col & 3);
}

// VE consecutive columns' sums of vector v.
template <int VE>
__device__ __forceinline__ void part_store(float* row, int v, int n, const float (&f)[VE]) {
  if constexpr (VE == 1) {
    row[v] = f[0];
  } else {
#pragma unroll
    for (int q = 0; q < VE / 4; ++q)
      *reinterpret_cast<float4*>(row + (static_cast<int64_t>(q) * (n / VE) + v) * 4) =
          make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  }
}

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

// Rows that are not whole vectors, in tensors that start on a vector: a row is
// taken as the vectors of memory that it touches, the first `shift` elements of
// which are not its own, and each of these is masked in the first and the last
// of them alone.  Rows `VE` apart have the same shift, so a CTA that takes only
// such rows keeps its threads' columns, and their parameters and sums in
// registers.
template <int VE>
struct Window {
  int n, shift, nvec;

  __device__ __forceinline__ Window(int64_t row, int n_)
      : n(n_),
        shift(static_cast<int>(row * n_) & (VE - 1)),
        nvec((n_ + shift + VE - 1) / VE) {}

  __device__ __forceinline__ int col(int v) const { return v * VE - shift; }  // of v's element 0
  __device__ __forceinline__ bool has(int col) const {
    return static_cast<unsigned>(col) < static_cast<unsigned>(n);
  }
  __device__ __forceinline__ bool cut(int v) const { return !has(col(v)) || !has(col(v) + VE - 1); }

  // vector v of the row whose window starts at `p`.  What is not the row's may be
  // anything: a neighbouring row's, or zeros in the tensor's last row, past
  // whose elements nothing is read.
  template <typename T>
  __device__ __forceinline__ Pack<T, VE> load(const T* p, int v, bool last) const {
    if (!last || !cut(v)) return ld_stream<T, VE>(p + static_cast<int64_t>(v) * VE);
    Pack<T, VE> out;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      out.v[e] = has(col(v) + e) ? p[static_cast<int64_t>(v) * VE + e] : from_f32<T>(0.0f);
    return out;
  }

  // zeros for what is not the row's
  template <typename T>
  __device__ __forceinline__ void mask(int v, Pack<T, VE>* f) const {
    if (!cut(v)) return;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (!has(col(v) + e)) f->v[e] = from_f32<T>(0.0f);
  }

  template <typename T>
  __device__ __forceinline__ void store(T* p, int v, const Pack<T, VE>& f) const {
    if (!cut(v)) return st_stream<T, VE>(p + static_cast<int64_t>(v) * VE, f);
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (has(col(v) + e)) p[static_cast<int64_t>(v) * VE + e] = f.v[e];
  }

  // the parameters of v's columns
  template <typename M>
  __device__ __forceinline__ Pack<M, VE> params(const M* p, int v) const {
    Pack<M, VE> out;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      out.v[e] = has(col(v) + e) ? __ldg(p + col(v) + e) : from_f32<M>(0.0f);
    return out;
  }
};

// ---------------------------------------------------------------------------
// Forward, the row in registers: read once, normalized, written once.
// ---------------------------------------------------------------------------
// Sum over the CTA with one barrier: every thread adds the warps' sums itself,
// in warp order.  `red` holds one float per warp; a later call on the same
// `red` needs a barrier between the two.
__device__ __forceinline__ float cta_sum_1b(float v, float* red) {
  v = warp_sum(v);
  const int nwarps = (blockDim.x + 31) >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < nwarps; ++w) t += red[w];
  return t;
}

// This thread's vectors first, first + step, ... (NV of them, below nvec) of
// one row: S formed, stored if wanted, and held.
template <typename T, typename M, int VE, int NV>
struct LayerRow {
  Pack<T, VE> s[NV];

  __device__ __forceinline__ void load(const LayerArgs<T, M>& a, int64_t base, int first, int step,
                                       int nvec) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      if (v < nvec) s[k] = ld_stream<T, VE>(a.x + base + static_cast<int64_t>(v) * VE);
    }
    if (!a.skip) return;
    Pack<T, VE> q[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      if (v < nvec) q[k] = ld_stream<T, VE>(a.skip + base + static_cast<int64_t>(v) * VE);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      if (v >= nvec) continue;
      float f[VE], kf[VE];
      unpack(s[k], f);
      unpack(q[k], kf);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], kf[e]);
      if (a.bias) {
        float bf[VE];
        ld_params<T, VE>(a.bias + static_cast<int64_t>(v) * VE, bf);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], bf[e]);
      }
      s[k] = pack_from<T, VE>(f);
      if (a.s) st_stream<T, VE>(a.s + base + static_cast<int64_t>(v) * VE, s[k]);
    }
  }

  __device__ __forceinline__ float sum(int first, int step, int nvec) const {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (first + k * step >= nvec) continue;
      float f[VE];
      unpack(s[k], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) t += f[e];
    }
    return t;
  }

  __device__ __forceinline__ float squares(float mu, int first, int step, int nvec) const {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (first + k * step >= nvec) continue;
      float f[VE];
      unpack(s[k], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = f[e] - mu;
        t = fmaf(d, d, t);
      }
    }
    return t;
  }

  __device__ __forceinline__ void store(const LayerArgs<T, M>& a, int64_t base, int first,
                                        int step, int nvec, float mu, float r) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      if (v >= nvec) continue;
      float f[VE], p[VE];
      unpack(s[k], f);
      ld_params<M, VE>(a.gamma + static_cast<int64_t>(v) * VE, p);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = (f[e] - mu) * r * p[e];
      if (a.beta) {
        ld_params<M, VE>(a.beta + static_cast<int64_t>(v) * VE, p);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] += p[e];
      }
      st_stream<T, VE>(a.y + base + static_cast<int64_t>(v) * VE, pack_from<T, VE>(f));
    }
  }
};

// Short rows: `tpr` <= 32 threads (a power of two) per row, both sums by
// butterflies over them, no barrier; persistent grid.
template <typename T, typename M, int VE, int NV>
__global__ void __launch_bounds__(256) layer_lane_kernel(const LayerArgs<T, M> a, int tpr,
                                                         int nvec) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, per = blockDim.x / tpr;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per; row0 < a.rows;
       row0 += static_cast<int64_t>(gridDim.x) * per) {
    const int64_t row = row0 + group;
    const int64_t base = row * a.n;
    const int nv = row < a.rows ? nvec : 0;  // the whole warp takes part in the sums
    LayerRow<T, M, VE, NV> x;
    if (nv) x.load(a, base, lane, tpr, nv);
    const float mu = seg_sum(x.sum(lane, tpr, nv), tpr) * a.inv_n;
    const float r = rsqrtf(fmaf(seg_sum(x.squares(mu, lane, tpr, nv), tpr), a.inv_n, a.eps));
    if (!nv) continue;
    x.store(a, base, lane, tpr, nv, mu, r);
    if (lane == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.inv_std) a.inv_std[row] = r;
    }
  }
}

// Longer rows: a CTA each, or a cluster of CTAs whose sums meet through
// distributed shared memory (tpr = threads of the cluster).
template <typename T, typename M, int VE, int NV>
__global__ void __launch_bounds__(kLayerThreads) layer_cta_kernel(const LayerArgs<T, M> a, int tpr,
                                                                  int nvec) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[2][16];
  __shared__ float slot[2];
  const unsigned csize = cluster_size();
  const unsigned rank = csize > 1 ? cluster_rank() : 0u;
  const int64_t row = blockIdx.x / csize, base = row * a.n;
  const int first = threadIdx.x + static_cast<int>(rank) * blockDim.x;
  LayerRow<T, M, VE, NV> x;
  x.load(a, base, first, tpr, nvec);
  float t = cta_sum_1b(x.sum(first, tpr, nvec), red[0]);
  if (csize > 1) t = cluster_sum(t, &slot[0], csize);
  const float mu = t * a.inv_n;
  t = cta_sum_1b(x.squares(mu, first, tpr, nvec), red[1]);
  if (csize > 1) t = cluster_sum(t, &slot[1], csize);
  const float r = rsqrtf(fmaf(t, a.inv_n, a.eps));
  x.store(a, base, first, tpr, nvec, mu, r);
  if (first == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.inv_std) a.inv_std[row] = r;
  }
  if (csize > 1) cluster_sync();  // peers may still read slot
}

// Rows that are not whole vectors, by windows: as above, but a CTA takes every
// `parts`-th row (a multiple of VE, or one row each).  Each thread keeps its
// columns' parameters in shared memory, where it alone reads them.
template <typename P>
__device__ __forceinline__ void keep16(uint4* at, int step, const P& p) {
  uint4 raw[sizeof(P) / 16];
  memcpy(raw, &p, sizeof(P));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(P) / 16); ++i) at[i * step] = raw[i];
}
template <typename P>
__device__ __forceinline__ P kept16(const uint4* at, int step) {
  uint4 raw[sizeof(P) / 16];
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(P) / 16); ++i) raw[i] = at[i * step];
  P p;
  memcpy(&p, raw, sizeof(P));
  return p;
}

// 16-byte pieces that a vector's gamma, beta and bias take
template <typename T, typename M, int VE>
__host__ __device__ constexpr int layer_window_pieces() {
  return 2 * (sizeof(Pack<M, VE>) / 16) + sizeof(Pack<T, VE>) / 16;
}

// What hides a row's latency is the other rows of the SM, so the registers are
// held to what lets five CTAs of 256 threads, or three (16-byte vectors of 16
// bits: 8192 x 4095 float16 takes 83.7 us, 91.0 without) or two (float32: 101,
// 133) of 512, be resident.
template <int VE, int NV>
constexpr int kLayerWindowThreads = NV == 1 || (VE == 4 && NV == 2) ? 256 : kLayerThreads;
template <int VE, int NV>
constexpr int kLayerWindowCtas = kLayerWindowThreads<VE, NV> == 256 ? 5 : VE == 4 ? 2 : 3;

template <typename T, typename M, int VE, int NV>
__global__ void __launch_bounds__(kLayerWindowThreads<VE, NV>, kLayerWindowCtas<VE, NV>)
layer_window_kernel(const LayerArgs<T, M> a, int tpr, int parts) {
  pdl_wait();
  pdl_trigger();
  using PM = Pack<M, VE>;
  using PT = Pack<T, VE>;
  extern __shared__ __align__(16) uint4 params[];
  __shared__ float red[2][16];
  __shared__ float slot[2];
  const unsigned csize = cluster_size();
  const unsigned rank = csize > 1 ? cluster_rank() : 0u;
  int64_t row = blockIdx.x / csize;
  const Window<VE> w(row, a.n);
  const int first = threadIdx.x + static_cast<int>(rank) * blockDim.x;
  const int lot = NV * blockDim.x;
  constexpr int kM = sizeof(PM) / 16;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = first + k * tpr;
    if (v >= w.nvec) continue;
    uint4* at = params + k * blockDim.x + threadIdx.x;
    keep16(at, lot, w.params(a.gamma, v));
    if (a.beta) keep16(at + kM * lot, lot, w.params(a.beta, v));
    if (a.bias) keep16(at + 2 * kM * lot, lot, w.params(a.bias, v));
  }
  for (; row < a.rows; row += parts) {
    const int64_t base = row * a.n - w.shift;
    const bool last = row == a.rows - 1;
    PT s[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * tpr;
      if (v < w.nvec) s[k] = w.load(a.x + base, v, last);
    }
    if (a.skip) {
      PT q[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * tpr;
        if (v < w.nvec) q[k] = w.load(a.skip + base, v, last);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * tpr;
        if (v >= w.nvec) continue;
        float f[VE], kf[VE];
        unpack(s[k], f);
        unpack(q[k], kf);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], kf[e]);
        if (a.bias) {
          unpack(kept16<PT>(params + 2 * kM * lot + k * blockDim.x + threadIdx.x, lot), kf);
#pragma unroll
          for (int e = 0; e < VE; ++e) f[e] = __fadd_rn(f[e], kf[e]);
        }
        s[k] = pack_from<T, VE>(f);
        if (a.s) w.store(a.s + base, v, s[k]);
      }
    }
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * tpr;
      if (v >= w.nvec) continue;
      w.mask(v, &s[k]);
      float f[VE];
      unpack(s[k], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) t += f[e];
    }
    t = cta_sum_1b(t, red[0]);
    if (csize > 1) t = cluster_sum(t, &slot[0], csize);
    const float mu = t * a.inv_n;
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * tpr;
      if (v >= w.nvec) continue;
      float f[VE];
      unpack(s[k], f);
      const bool cut = w.cut(v);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = f[e] - mu;
        if (!cut || w.has(w.col(v) + e)) t = fmaf(d, d, t);
      }
    }
    t = cta_sum_1b(t, red[1]);
    if (csize > 1) t = cluster_sum(t, &slot[1], csize);
    const float r = rsqrtf(fmaf(t, a.inv_n, a.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * tpr;
      if (v >= w.nvec) continue;
      const uint4* at = params + k * blockDim.x + threadIdx.x;
      float f[VE], p[VE];
      unpack(s[k], f);
      unpack(kept16<PM>(at, lot), p);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = (f[e] - mu) * r * p[e];
      if (a.beta) {
        unpack(kept16<PM>(at + kM * lot, lot), p);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] += p[e];
      }
      w.store(a.y + base, v, pack_from<T, VE>(f));
    }
    if (first == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.inv_std) a.inv_std[row] = r;
    }
  }
  if (csize > 1) cluster_sync();  // peers may still read slot
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
  const unsigned nvec = a.n / VE;  // unsigned: v passes 2^31 past the longest rows
  float sum = 0.0f;
  for (unsigned v = threadIdx.x; v < nvec; v += blockDim.x) {
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
  for (unsigned v = threadIdx.x; v < nvec; v += blockDim.x) {
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
  for (unsigned v = threadIdx.x; v < nvec; v += blockDim.x) {
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

// ---------------------------------------------------------------------------
// Gradient in one pass: a row's g = dy * gamma and u = (S - mu) * r are held in
// registers, its two means reduced, dS written, and the row added to the column
// sums that the threads hold for their own columns.  Each input is read once.
// At the copy bandwidth an SM's schedulers have about 45 issue slots per 32
// elements, so the arithmetic goes two elements at a time.  Every product and
// sum is rounded by itself, so that every instantiation gives the same bits.
// ---------------------------------------------------------------------------
// Vectors a thread holds at most: sixteen elements, whose sums and row fit 128 registers.
template <int VE>
__host__ __device__ constexpr int layer_grad_most() {
  return VE == 8 ? 2 : VE == 4 ? 4 : 8;
}

template <typename T, typename M, int VE, int NV, bool BIAS>
struct LayerGradRow {
  using V = typename std::conditional<VE == 1, float, float2>::type;  // pairs of a vector
  static constexpr int H = (VE + 1) / 2;
  V dg[NV][H] = {}, db[NV][H] = {}, dc[BIAS ? NV : 1][H] = {};
  V gm[NV][H];
  V g[NV][H], u[NV][H];

  __device__ __forceinline__ static V at(const Pack<T, VE>& p, int i) {
    if constexpr (VE == 1) return to_f32(p.v[0]);
    else return get2(p, i);
  }

  // gamma of this thread's columns: vectors first, first + step, ... below nvec
  __device__ __forceinline__ void load_gamma(const M* gamma, int first, int step, int nvec) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      float f[VE] = {};
      if (v < nvec) ld_params<M, VE>(gamma + static_cast<int64_t>(v) * VE, f);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if constexpr (VE == 1) gm[k][i] = f[0];
        else gm[k][i] = make_float2(f[2 * i], f[2 * i + 1]);
      }
    }
  }

  // the same by windows
  __device__ __forceinline__ void load_gamma(const M* gamma, const Window<VE>& w, int first,
                                             int step, int end) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      float f[VE] = {};
      if (v < end) unpack(w.params(gamma, v), f);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if constexpr (VE == 1) gm[k][i] = f[0];
        else gm[k][i] = make_float2(f[2 * i], f[2 * i + 1]);
      }
    }
  }

  // vector k of a row: adds it to dgamma and dbeta, and to the sums of g (tg)
  // and g * u (tu)
  __device__ __forceinline__ void take(int k, const Pack<T, VE>& dy, const Pack<T, VE>& s,
                                       float mu, float r, V& tg, V& tu) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const V d = at(dy, i);
      u[k][i] = mul2(add2(at(s, i), every<V>(-mu)), every<V>(r));
      g[k][i] = mul2(d, gm[k][i]);
      dg[k][i] = fma2(d, u[k][i], dg[k][i]);
      db[k][i] = add2(db[k][i], d);
      tg = add2(tg, g[k][i]);
      tu = fma2(g[k][i], u[k][i], tu);
    }
  }

  // dS of vector k, k1 = -r * mean(g), k2 = -r * mean(g * u)
  __device__ __forceinline__ Pack<T, VE> give(int k, float r, float k1, float k2,
                                              const Pack<T, VE>* ds) {
    Pack<T, VE> out;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      V d = fma2(g[k][i], every<V>(r), fma2(u[k][i], every<V>(k2), every<V>(k1)));
      if (ds) d = add2(d, at(*ds, i));
      if constexpr (BIAS) dc[k][i] = add2(dc[k][i], d);
      if constexpr (VE == 1) out.v[0] = from_f32<T>(d);
      else set2(out, i, d.x, d.y);
    }
    return out;
  }

  // one of dg, db and dc of a vector, an element at a time
  __device__ __forceinline__ static void elements(const V (&p)[H], float (&f)[VE]) {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if constexpr (VE == 1) f[0] = p[0];
      else f[e] = e % 2 ? p[e / 2].y : p[e / 2].x;
    }
  }
};

// One tensor's bytes of a tile: `len` elements from element `off` on, copied to
// `dst` from the 16-byte boundary below them on (a bulk copy starts and ends on
// such boundaries).  The copy may take bytes of neighbouring rows, but none
// outside the tensor: what it leaves out at the tensor's ends, take() reads from
// global memory.
template <typename T, int VE>
struct TileBytes {
  const T* p;         // element `off`
  uintptr_t lo, hi;   // what is copied
  int shift;          // bytes from dst to element `off`

  __device__ __forceinline__ TileBytes(const T* tensor, int64_t numel, int64_t off, int64_t len)
      : p(tensor + off) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if constexpr (VE > 1) {  // whole vectors
      shift = 0;
      lo = a;
      hi = a + len * sizeof(T);
    } else {
      shift = static_cast<int>(a & 15);
      const uintptr_t begin = (reinterpret_cast<uintptr_t>(tensor) + 15) & ~uintptr_t{15};
      const uintptr_t end = reinterpret_cast<uintptr_t>(tensor + numel) & ~uintptr_t{15};
      lo = a & ~uintptr_t{15};
      hi = (a + len * sizeof(T) + 15) & ~uintptr_t{15};
      if (lo < begin) lo = begin;
      if (hi > end) hi = end;
      if (hi < lo) hi = lo;
    }
  }

  __device__ __forceinline__ unsigned bytes() const { return static_cast<unsigned>(hi - lo); }

  __device__ __forceinline__ void copy(unsigned char* dst, unsigned long long* bar) const {
    if (hi > lo)
      bulk_load(dst + (lo - (reinterpret_cast<uintptr_t>(p) - shift)),
                reinterpret_cast<const void*>(lo), bytes(), bar);
  }

  // vector v of the tile
  __device__ __forceinline__ Pack<T, VE> take(const unsigned char* dst, int v, bool edge) const {
    if constexpr (VE == 1) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p + v);
      if (edge && (at < lo || at >= hi)) return ld_stream<T, 1>(p + v);
    }
    return *reinterpret_cast<const Pack<T, VE>*>(dst + shift + v * static_cast<int>(sizeof(T)) * VE);
  }
};

// At the end of a lane kernel the row groups of a warp add their column sums by
// butterflies, then the warps theirs through shared memory, in warp order.
constexpr int kLayerGradLaneThreads = 256;
template <typename T, typename M, int VE, int NV, bool BIAS>
__device__ __forceinline__ void layer_grad_lane_sums(
    const LayerGradArgs<T, M>& a, const LayerGradRow<T, M, VE, NV, BIAS>& x,
    float (*acc)[32 * NV * VE], int tpr) {
  constexpr int kOut = BIAS ? 3 : 2;
  const int lane = threadIdx.x & (tpr - 1);
  for (int w = 0; w < kLayerGradLaneThreads / 32; ++w) {
    if (threadIdx.x / 32 == w) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float fg[VE], fb[VE], fc[VE];
        x.elements(x.dg[k], fg);
        x.elements(x.db[k], fb);
        x.elements(x.dc[BIAS ? k : 0], fc);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float g = fg[e], b = fb[e], c = fc[e];
          for (int o = tpr; o < 32; o *= 2) {
            g += __shfl_xor_sync(0xffffffffu, g, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
            if constexpr (BIAS) c += __shfl_xor_sync(0xffffffffu, c, o);
          }
          const int col = (lane + k * tpr) * VE + e;
          if ((threadIdx.x & 31) < tpr) {
            acc[0][col] = w ? acc[0][col] + g : g;
            acc[1][col] = w ? acc[1][col] + b : b;
            if constexpr (BIAS) acc[kOut - 1][col] = w ? acc[kOut - 1][col] + c : c;
          }
        }
      }
    }
    __syncthreads();
  }
  float* p = a.part + blockIdx.x * 3 * a.pitch;
  for (int col = threadIdx.x; col < a.n; col += kLayerGradLaneThreads) {
#pragma unroll
    for (int o = 0; o < kOut; ++o) p[o * a.pitch + part_at(col, a.n, VE)] = acc[o][col];
  }
}

// Writes v at `local`'s place in CTA `rank` of the cluster; its 8 bytes complete on
// the barrier at `bar`'s place there.
__device__ __forceinline__ void send_to_peer(float2* local, unsigned rank, float2 v,
                                             unsigned long long* bar) {
  unsigned to, at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
               :: "r"(to), "f"(v.x), "f"(v.y), "r"(at) : "memory");
}

// The inputs are streamed through shared memory: one thread keeps the next
// `stages` tiles of dy, S and ds (contiguous bytes, one bulk copy each) on their
// way while the CTA works on the present one.  Without the stream, threads can
// hold no more than the present row in flight and stand still for its two means
// (16384 x 4096 bfloat16: 135 us).  Part p takes tiles p, p + parts, ....
//
// A tile is a row (of a cluster's CTA: its slice of the row), or with LANE the
// 256 / tpr consecutive rows that the CTA's lane groups take.  The CTAs of a
// cluster send their sums of a row to one another (4096 x 16384 bfloat16: 120 us,
// 173 with a cluster barrier and remote loads); two sets of slots are enough, for
// a CTA sends its sums of the next row only once it has all of this one.
//
// A stage is free again once the CTA has met at the next tile's barrier.  The waits
// for a copy and for the other CTAs' sums are bounded; a thread whose wait gave up
// records it and runs on without waiting (its outputs are then undefined), so that
// every barrier is met.
//
// With WINDOW rows are taken by windows: a part's rows are then a multiple of VE
// apart.
constexpr int kLayerStages = 4;  // at most; 2 where that lets an SM hold two CTAs
constexpr unsigned long long kLayerLimitNs = 1000000000ull;
// what a test leaves out, so that the waits for it give up
enum LayerStall { kLayerNoCopies = 1, kLayerNoSums = 2 };

template <typename T, int VE>
__host__ __device__ constexpr int layer_slot_bytes(int vectors) {
  return VE > 1 ? vectors * 16 : (vectors * static_cast<int>(sizeof(T)) + 15) / 16 * 16 + 16;
}

template <typename T, typename M, int VE, int NV, bool BIAS, bool LANE, bool WINDOW = false>
__global__ void __launch_bounds__(LANE ? kLayerGradLaneThreads : kLayerThreads, 1)
layer_grad_ring_kernel(const LayerGradArgs<T, M> a, int tpr, int nvec, int slice, int stages,
                       unsigned* status, unsigned long long limit_ns, int stall) {
  using P = Pack<T, VE>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ alignas(8) unsigned long long full[kLayerStages];
  __shared__ float2 red[2][16];
  __shared__ float2 slot[2][8];
  __shared__ alignas(8) unsigned long long sent[2];
  __shared__ float acc[LANE ? (BIAS ? 3 : 2) : 1][LANE ? 32 * NV * VE : 1];
  // only slices that take every vector a thread can hold are parts of longer rows
  const unsigned csize = !LANE && NV == layer_grad_most<VE>() ? cluster_size() : 1u;
  const unsigned rank = csize > 1 ? cluster_rank() : 0u;
  const int part = blockIdx.x / csize;
  const Window<VE> w(part, a.n);
  const int shift = WINDOW ? w.shift : 0;
  if (WINDOW) nvec = w.nvec;
  // this CTA's vectors of a row: [lo, lo + count)
  const int lo = static_cast<int>(rank) * slice;
  const int count = LANE ? nvec : (nvec - lo < slice ? (nvec > lo ? nvec - lo : 0) : slice);
  const int rows_per = LANE ? kLayerGradLaneThreads / tpr : 1;
  const int first = LANE ? threadIdx.x & (tpr - 1) : threadIdx.x;
  const int step = LANE ? tpr : blockDim.x;
  const int group = LANE ? threadIdx.x / tpr : 0;
  const int tiles_all = static_cast<int>((a.rows + rows_per - 1) / rows_per);
  const int tiles = tiles_all > part ? (tiles_all - part + a.parts - 1) / a.parts : 0;
  const int slot_bytes = layer_slot_bytes<T, VE>(rows_per * slice);
  const int64_t stride = static_cast<int64_t>(a.parts) * rows_per;  // rows from tile to tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kLayerStages; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sent[i], 1);
    mbar_init_fence();
  }
  if (csize > 1) cluster_sync();  // peers complete on `sent`
  else __syncthreads();
  pdl_wait();
  pdl_trigger();

  // the tile whose first row is `row`: its place in the tensors, its elements
  auto offset = [&](int64_t row) { return row * a.n - shift + static_cast<int64_t>(lo) * VE; };
  auto length = [&](int64_t row) {
    return static_cast<int>(a.rows - row < rows_per ? a.rows - row : rows_per) * count * VE;
  };
  auto issue = [&](int64_t row, int st) {  // thread 0: that tile into stage st
    const int64_t off = offset(row);
    const int len = length(row);
    unsigned char* dst = ring + st * 3 * slot_bytes;
    unsigned long long* bar = &full[st];
    if constexpr (VE > 1) {
      unsigned bytes = len * static_cast<unsigned>(sizeof(T));
      if constexpr (WINDOW) {  // the tensor's last vector may not be whole
        const int64_t left = (a.rows * a.n - off) / VE;
        if (left < count) bytes = left > 0 ? static_cast<unsigned>(left) * 16 : 0u;
      }
      mbar_arrive_expect_tx(bar, bytes * (a.ds ? 3 : 2));
      if (bytes == 0) return;
      bulk_load(dst, a.dy + off, bytes, bar);
      bulk_load(dst + slot_bytes, a.s + off, bytes, bar);
      if (a.ds) bulk_load(dst + 2 * slot_bytes, a.ds + off, bytes, bar);
    } else {
      const int64_t numel = a.rows * a.n;
      const TileBytes<T, VE> dy(a.dy, numel, off, len), s(a.s, numel, off, len),
          ds(a.ds ? a.ds : a.s, numel, off, len);
      mbar_arrive_expect_tx(bar, dy.bytes() + s.bytes() + (a.ds ? ds.bytes() : 0u));
      dy.copy(dst, bar);
      s.copy(dst + slot_bytes, bar);
      if (a.ds) ds.copy(dst + 2 * slot_bytes, bar);
    }
  };
  const int64_t row0 = static_cast<int64_t>(part) * rows_per;
  if (threadIdx.x == 0)
    for (int i = 0; i < stages && i < tiles && stall != kLayerNoCopies; ++i) issue(row0 + i * stride, i);

  // vector v of a stage, cut to the row's elements; the tensor's last elements,
  // which no copy brings, come from global memory
  auto at_edge = [&](const T* window, const P* staged, int v, bool last) {
    P p = last ? w.load(window, lo + v, true) : staged[v];
    w.mask(lo + v, &p);
    return p;
  };
  LayerGradRow<T, M, VE, NV, BIAS> x;
  if constexpr (WINDOW) x.load_gamma(a.gamma, w, lo + first, step, lo + count);
  else x.load_gamma(a.gamma + static_cast<int64_t>(lo) * VE, first, step, count);
  bool alive = true;
  int64_t row = row0 + group;
  // the next row's statistics are on their way as well
  float mu_next = 0.0f, r_next = 0.0f;
  if (row < a.rows) {
    mu_next = a.mean[row];
    r_next = a.inv_std[row];
  }
  int st = 0, before = 0;
  unsigned parity = 0;
  for (int i = 0; i < tiles; ++i) {
    const int nv = row < a.rows ? count : 0;
    const float mu = mu_next, r = r_next;
    if (row + stride < a.rows) {
      mu_next = a.mean[row + stride];
      r_next = a.inv_std[row + stride];
    }
    const unsigned char* stage = ring + st * 3 * slot_bytes;
    if (alive && !mbar_wait(&full[st], parity, limit_ns)) {
      alive = false;
      atomicExch(status, kStatusDeviceTimeout);
    }
    using V = typename LayerGradRow<T, M, VE, NV, BIAS>::V;
    V tg = every<V>(0.0f), tu = tg;
    if constexpr (VE > 1) {
      const P* dy = reinterpret_cast<const P*>(stage) + group * count;
      const P* s = reinterpret_cast<const P*>(stage + slot_bytes) + group * count;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * step;
        if (v >= nv) continue;
        if (WINDOW && w.cut(lo + v)) {
          const int64_t off = row * a.n - shift;
          const bool last = row == a.rows - 1;
          x.take(k, at_edge(a.dy + off, dy, v, last), at_edge(a.s + off, s, v, last), mu, r, tg,
                 tu);
        } else {
          x.take(k, dy[v], s[v], mu, r, tg, tu);
        }
      }
    } else {
      const int64_t numel = a.rows * a.n, off = offset(row - group);
      const int len = length(row - group);
      const bool edge = off == 0 || off + len + 8 >= numel;  // copies may be cut short there
      const TileBytes<T, VE> dy(a.dy, numel, off, len), s(a.s, numel, off, len);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * step, at = group * count + v;
        if (v < nv)
          x.take(k, dy.take(stage, at, edge), s.take(stage + slot_bytes, at, edge), mu, r, tg, tu);
      }
    }
    float2 t = make_float2(total(tg), total(tu));
    if constexpr (LANE) {
      t.x = seg_sum(t.x, tpr);
      t.y = seg_sum(t.y, tpr);
      __syncthreads();
    } else {
      t = cta_sum2_1b(t, red[i & 1]);
    }
    // everyone is done with the tile before this one
    if (threadIdx.x == 0 && alive && i > 0 && i - 1 + stages < tiles)
      issue(row - group + (stages - 1) * stride, before);
    if (csize > 1) {
      const int b = i & 1;
      // after a wait that gave up nothing is armed or sent, and the peers give up too
      if (threadIdx.x == 0 && alive) mbar_arrive_expect_tx(&sent[b], csize * 8);
      if (threadIdx.x < csize && alive && stall != kLayerNoSums)
        send_to_peer(&slot[b][rank], threadIdx.x, t, &sent[b]);
      if (alive && !mbar_wait(&sent[b], i >> 1 & 1, limit_ns)) {
        alive = false;
        atomicExch(status, kStatusDeviceTimeout);
      }
      t = slot[b][0];
      for (unsigned q = 1; q < csize; ++q) {
        t.x += slot[b][q].x;
        t.y += slot[b][q].y;
      }
    }
    const float k1 = -r * (t.x * a.inv_n), k2 = -r * (t.y * a.inv_n);
    T* dx = a.dx ? a.dx + offset(row) : nullptr;
    if constexpr (VE > 1) {
      const P* ds = reinterpret_cast<const P*>(stage + 2 * slot_bytes) + group * count;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * step;
        if (v >= nv) continue;
        if (WINDOW && w.cut(lo + v)) {
          const int64_t off = row * a.n - shift;
          P h;
          if (a.ds) h = at_edge(a.ds + off, ds, v, row == a.rows - 1);
          const P out = x.give(k, r, k1, k2, a.ds ? &h : nullptr);
          if (dx) w.store(a.dx + off, lo + v, out);
        } else {
          const P out = x.give(k, r, k1, k2, a.ds ? ds + v : nullptr);
          if (dx) st_stream<T, VE>(dx + v * VE, out);
        }
      }
    } else {
      const int64_t numel = a.rows * a.n, off = offset(row - group);
      const int len = length(row - group);
      const bool edge = off == 0 || off + len + 8 >= numel;
      const TileBytes<T, VE> ds(a.ds ? a.ds : a.s, numel, off, len);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * step;
        if (v >= nv) continue;
        Pack<T, VE> h;
        if (a.ds) h = ds.take(stage + 2 * slot_bytes, group * count + v, edge);
        const Pack<T, VE> out = x.give(k, r, k1, k2, a.ds ? &h : nullptr);
        if (dx) st_stream<T, VE>(dx + v, out);
      }
    }
    row += stride;
    before = st;
    if (++st == stages) {
      st = 0;
      parity ^= 1;
    }
  }
  if (!alive && threadIdx.x == 0 && stall != kLayerNoCopies)  // copies still in flight land before the CTA ends
    for (int i = 0; i < stages; ++i) {
      mbar_wait(&full[i], 0, limit_ns);
      mbar_wait(&full[i], 1, limit_ns);
    }
  const bool sums = a.dgamma || a.dbeta || a.dbias;
  if constexpr (LANE) {
    if (sums) layer_grad_lane_sums<T, M, VE, NV, BIAS>(a, x, acc, tpr);
  } else if constexpr (WINDOW) {
    // through shared memory, where they are turned to their columns' order
    float* turn = reinterpret_cast<float*>(ring);
    float* p = a.part + part * 3 * a.pitch;
    for (int o = 0; o < (BIAS ? 3 : 2) && sums; ++o) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = first + k * step;
        if (v >= count) continue;
        float f[VE];
        x.elements(o == 0 ? x.dg[k] : o == 1 ? x.db[k] : x.dc[BIAS ? k : 0], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) turn[v * VE + e] = f[e];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < count * VE; i += blockDim.x) {
        const int col = w.col(lo) + i;
        if (w.has(col)) p[o * a.pitch + col] = turn[i];
      }
    }
  } else {
    float* p = a.part + part * 3 * a.pitch;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = first + k * step;
      if (v >= count || !sums) continue;
      float f[VE];
      x.elements(x.dg[k], f);
      part_store<VE>(p, lo + v, a.n, f);
      x.elements(x.db[k], f);
      part_store<VE>(p + a.pitch, lo + v, a.n, f);
      if constexpr (BIAS) {
        x.elements(x.dc[k], f);
        part_store<VE>(p + 2 * a.pitch, lo + v, a.n, f);
      }
    }
  }
  if (csize > 1) {
    cluster_sync();  // peers' sums may still be on their way to this CTA
    if (!alive && threadIdx.x == 0)
      for (int i = 0; i < 2 && i < tiles; ++i)
        mbar_wait(&sent[(tiles - 1 - i) & 1], (tiles - 1 - i) >> 1 & 1, limit_ns);
  }
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
  const unsigned nvec = a.n / VE;  // unsigned: v passes 2^31 past the longest rows
  const float mu = a.mean[row], r = a.inv_std[row];
  float2 acc = make_float2(0.0f, 0.0f);
  for (unsigned v = threadIdx.x; v < nvec; v += blockDim.x) {
    const int64_t off = base + static_cast<int64_t>(v) * VE;
    float dy[VE], s[VE], gm[VE];
    unpack(ld_reuse<T, VE>(a.dy + off), dy);
    unpack(ld_reuse<T, VE>(a.s + off), s);
    ld_params<M, VE>(a.gamma + static_cast<int64_t>(v) * VE, gm);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float g = __fmul_rn(dy[e], gm[e]);
      acc.x += g;
      acc.y = fmaf(g, __fmul_rn(s[e] - mu, r), acc.y);
    }
  }
  acc = cta_sum2(acc, red);
  const float c1 = acc.x * a.inv_n, c2 = acc.y * a.inv_n;
  if (threadIdx.x == 0) a.coef[row] = make_float2(c1, c2);
  if (!a.dx) return;
  const float k1 = -r * c1, k2 = -r * c2;
  for (unsigned v = threadIdx.x; v < nvec; v += blockDim.x) {
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
#pragma unroll
    for (int e = 0; e < VE; ++e) d[e] = fmaf(g[e], r, fmaf(u[e], k2, k1));
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
  float* p = a.part + part * 3 * a.pitch + col;
  p[0] = dg;
  p[a.pitch] = db;
  if (a.dbias) p[2 * a.pitch] = dc;
}

// The parts' sums added in a fixed order: a CTA takes COLS columns of one of the
// three outputs, COLS / 4 threads (16 bytes each) a part's columns; then warps,
// then the CTA, add theirs.  Few columns per CTA keep more of the device at work
// on rows of few columns (16384 x 768 bfloat16: the gradient takes 26.2 us with
// 32, 28.0 with 128); rows of many give enough CTAs, and the wider ones take less
// (64 x 4096: 5.5 us, 6.6 with 32).
template <int COLS>
constexpr int kLayerFinishThreads = COLS == 32 ? 512 : 1024;
template <typename T, typename M, int COLS>
__global__ void __launch_bounds__(kLayerFinishThreads<COLS>)
layer_grad_finish_kernel(const LayerGradArgs<T, M> a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kThreads = kLayerFinishThreads<COLS>, kWide = COLS / 4;
  __shared__ float4 red[kThreads / 32][kWide];
  const int which = blockIdx.y;
  if (which == 0 ? !a.dgamma : which == 1 ? !a.dbeta : !a.dbias) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * COLS + lane % kWide * 4;
  const float* src = a.part + which * a.pitch + at;
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (at < a.pitch) {  // what pads a row out to whole vectors is not used
#pragma unroll 8
    for (int p = threadIdx.x / kWide; p < a.parts; p += kThreads / kWide) {
      const float4 v = *reinterpret_cast<const float4*>(src + p * 3 * a.pitch);
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
  }
#pragma unroll
  for (int o = kWide; o < 32; o *= 2) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
    t.w += __shfl_xor_sync(0xffffffffu, t.w, o);
  }
  if (lane < kWide) red[warp][lane] = t;
  __syncthreads();
  const int64_t from = static_cast<int64_t>(blockIdx.x) * COLS + threadIdx.x;
  if (threadIdx.x >= COLS || from >= a.n) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += reinterpret_cast<const float*>(red[w])[threadIdx.x];
  // the column that lies there (part_at)
  int64_t out = from;
  if (a.ve == 8) {
    const int64_t q = from / 4, plane = q >= a.n / 8 ? 1 : 0;
    out = (q - plane * (a.n / 8)) * 8 + plane * 4 + from % 4;
  }
  if (which == 0) a.dgamma[out] = from_f32<M>(sum);
  else if (which == 1) a.dbeta[out] = from_f32<M>(sum);
  else a.dbias[out] = from_f32<T>(sum);
}

}  // namespace b200norm
