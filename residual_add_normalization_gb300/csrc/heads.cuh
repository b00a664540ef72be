// heads.cuh -- query and key heads on the way to attention: rotation of pairs of
// elements by the token's position, with or without an RMS norm of the head before
// it, and the gradients (sm_103a).
//
// With the pair (a, b) of a head, its frequency f and the token's position p:
//   (a, b) -> (a c - b s, b c + a s),  c = scale cos(p f), s = scale sin(p f);
// the norm before it is u = x r, r = 1 / sqrt(mean(x^2) + eps), a = u gamma.
//
// Bound by HBM: a head is read once and written once.  A row (one head of one token)
// is held by a group of lanes in registers; a lane holds both halves of its pairs, so
// the rotation needs no exchange: its unit is two accesses, u and u + rot / 2 in the
// half layout, neighbours otherwise.  A warp takes one token (or a part of its heads)
// and walks the heads, so that a pair's cosine and sine are made once a token.
//
// Angles: a frequency is kept as turns per position in units of 2^-64, so that the
// low 64 bits of position * frequency are the angle without its whole turns, exactly:
// positions cost no digits, and no binary64 operation is made per token.
#pragma once

#include "common.cuh"
#include "heads.h"

namespace b200norm {

constexpr int kHeadWarps = 8;

struct HeadsArgs {
  HeadsCall c;
  unsigned tokens, seq;
  int units, lanes;
  int steps[2];    // per token: the heads in groups of 32 / lanes
  int splits;      // parts of a token's steps, a warp each
  int parts[2];    // gradient: CTAs of queries and of keys
};

// -- angles -----------------------------------------------------------------------

// Radians per position to turns per position, mod 1, in units of 2^-64.
__device__ __forceinline__ unsigned long long phase_step(double radians) {
  constexpr double kInv2Pi = 0.15915494309189535;
  double t = radians * kInv2Pi;
  t -= floor(t);
  return __double2ull_rz(t * 18446744073709551616.0);
}

// Cosine and sine of `phase` 2^-32 turns: the nearest quarter turn is taken off
// exactly, and on the eighth of a turn that is left to either side (|a| <= pi / 4) the
// Taylor series end below 2.5e-8.
__device__ __forceinline__ void phase_cos_sin(unsigned phase, float& c, float& s) {
  constexpr float kTurn = 1.4629180792671596e-9f;  // 2 pi / 2^32
  const unsigned quarter = (phase + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int>(phase - (quarter << 30))) * kTurn;
  const float q = a * a;
  float sn = fmaf(q, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
  sn = fmaf(sn, q, 8.3333333e-3f);
  sn = fmaf(sn, q, -1.6666667e-1f);
  sn = fmaf(sn * q, a, a);
  float cs = fmaf(q, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!, 1/6!, 1/4!
  cs = fmaf(cs, q, -1.3888889e-3f);
  cs = fmaf(cs, q, 4.1666667e-2f);
  cs = fmaf(cs, q, -0.5f);
  cs = fmaf(cs, q, 1.0f);
  const bool swap = quarter & 1;
  const float x = swap ? sn : cs, y = swap ? cs : sn;
  c = (quarter + 1) & 2 ? -x : x;  // quarters 1 and 2
  s = quarter & 2 ? -y : y;        // quarters 2 and 3
}

// -- rows -------------------------------------------------------------------------

// Where a lane's units lie: elements lo.. and hi.. of the row, VE each.
template <int VE, int K>
struct HeadUnits {
  int lo[K], hi[K];    // element of the row, -1: none
  int pair[K];         // first of the unit's VE pairs
};

template <int VE, int K>
__device__ __forceinline__ HeadUnits<VE, K> head_units(const HeadsArgs& g, int sub) {
  HeadUnits<VE, K> u;
  const int half = g.c.interleaved ? 0 : g.c.rot / 2;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = sub + k * g.lanes;
    const bool in = i < g.units;
    u.pair[k] = i * VE;
    if (i * VE < half) {
      u.lo[k] = in ? i * VE : -1;
      u.hi[k] = in ? i * VE + half : -1;
    } else {
      u.lo[k] = in ? 2 * i * VE : -1;
      u.hi[k] = in && 2 * i * VE + VE < g.c.size ? 2 * i * VE + VE : -1;
    }
  }
  return u;
}

template <typename T, int VE, int K>
struct HeadRow {
  Pack<T, VE> lo[K], hi[K];
};

template <typename T, int VE, int K>
__device__ __forceinline__ void head_load(HeadRow<T, VE, K>& r, const T* p, bool in,
                                          const HeadUnits<VE, K>& u) {
  const Pack<T, VE> zero = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    r.lo[k] = in && u.lo[k] >= 0 ? ld_stream<T, VE>(p + u.lo[k]) : zero;
    r.hi[k] = in && u.hi[k] >= 0 ? ld_stream<T, VE>(p + u.hi[k]) : zero;
  }
}

template <typename T, int VE, int K>
__device__ __forceinline__ void head_store(T* p, bool in, const HeadUnits<VE, K>& u,
                                           const float (&lo)[K][VE], const float (&hi)[K][VE]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (in && u.lo[k] >= 0) st_stream<T, VE>(p + u.lo[k], pack_from<T, VE>(lo[k]));
    if (in && u.hi[k] >= 0) st_stream<T, VE>(p + u.hi[k], pack_from<T, VE>(hi[k]));
  }
}

// Cosine and sine (scaled, the sine's sign turned for the inverse) of a lane's pairs.
template <int VE, int K>
struct HeadAngles {
  float c[K][VE], s[K][VE];
};

template <int VE, int K>
__device__ __forceinline__ void head_angles(const HeadsArgs& g, const unsigned long long* steps,
                                            const HeadUnits<VE, K>& u, unsigned b, unsigned t,
                                            float sine, HeadAngles<VE, K>& a) {
  const int pairs = g.c.rot / 2;
  if (pairs == 0) return;
  const int64_t at = b * g.c.pos_batch + t * g.c.pos_token;
  const long long p = g.c.pos64 ? static_cast<const long long*>(g.c.positions)[at]
                                : static_cast<const int*>(g.c.positions)[at];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const int n = u.pair[k] + i;
      const unsigned long long phase =
          static_cast<unsigned long long>(p) * steps[n < pairs ? n : 0];
      phase_cos_sin(static_cast<unsigned>(phase >> 32), a.c[k][i], a.s[k][i]);
      a.c[k][i] *= g.c.scale;
      a.s[k][i] *= sine;
    }
}

// The pairs of a unit turned; elements past rot stay as they are.
template <int VE>
__device__ __forceinline__ void turn(const HeadsArgs& g, int pair, const float (&c)[VE],
                                     const float (&s)[VE], float (&lo)[VE], float (&hi)[VE]) {
  const int pairs = g.c.rot / 2;
  if (pair >= pairs) return;
  if (VE == 1 || !g.c.interleaved) {  // all of the unit's pairs, each across lo and hi
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float a = lo[i], b = hi[i];
      lo[i] = fmaf(a, c[i], -(b * s[i]));
      hi[i] = fmaf(b, c[i], a * s[i]);
    }
    return;
  }
  if constexpr (VE > 1) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (pair + i >= pairs) continue;
      float& x = i < VE / 2 ? lo[2 * i] : hi[2 * i - VE];
      float& y = i < VE / 2 ? lo[2 * i + 1] : hi[2 * i + 1 - VE];
      const float a = x, b = y;
      x = fmaf(a, c[i], -(b * s[i]));
      y = fmaf(b, c[i], a * s[i]);
    }
  }
}

// What a CTA's rows share, in shared memory: turns per position, and gamma widened.
struct HeadShared {
  unsigned long long steps[kMaxHeadSize / 2];
  alignas(16) float gamma[2][kMaxHeadSize];
};

__device__ __forceinline__ void head_shared(const HeadsArgs& g, HeadShared& sh) {
  for (int i = threadIdx.x; i < g.c.rot / 2; i += blockDim.x)
    sh.steps[i] = phase_step(__ldg(g.c.inv_freq + i));
  if (g.c.norm) {
    for (int i = threadIdx.x; i < 2 * g.c.size; i += blockDim.x) {
      const int n = i >= g.c.size, j = i - n * g.c.size;
      const void* p = g.c.set[n].gamma;
      float v = 1.0f;
      if (p && g.c.set[n].heads > 0) {
        v = g.c.m == DType::F32   ? static_cast<const float*>(p)[j]
            : g.c.m == DType::F16 ? to_f32(static_cast<const __half*>(p)[j])
                                  : to_f32(static_cast<const __nv_bfloat16*>(p)[j]);
      }
      sh.gamma[n][j] = v;
    }
  }
  __syncthreads();
}

template <int VE, int K>
__device__ __forceinline__ void head_gamma(const float* gamma, const HeadUnits<VE, K>& u,
                                           float (&lo)[K][VE], float (&hi)[K][VE]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      lo[k][i] = u.lo[k] >= 0 ? gamma[u.lo[k] + i] : 0.0f;
      hi[k][i] = u.hi[k] >= 0 ? gamma[u.hi[k] + i] : 0.0f;
    }
}

// -- forward ----------------------------------------------------------------------

template <typename T, int VE, int K, bool NORM>
__global__ void __launch_bounds__(32 * kHeadWarps) heads_kernel(const HeadsArgs g) {
  __shared__ HeadShared sh;
  pdl_wait();
  pdl_trigger();
  head_shared(g, sh);
  const int lane = threadIdx.x & 31;
  const int sub = lane & (g.lanes - 1), row = lane / g.lanes, rows = 32 / g.lanes;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kHeadWarps + (threadIdx.x >> 5);
  const unsigned token = static_cast<unsigned>(item / g.splits);
  if (token >= g.tokens) return;
  const int split = static_cast<int>(item - static_cast<int64_t>(token) * g.splits);
  const unsigned b = token / g.seq, t = token - b * g.seq;
  const HeadUnits<VE, K> u = head_units<VE, K>(g, sub);
  HeadAngles<VE, K> angle;
  head_angles<VE, K>(g, sh.steps, u, b, t, g.c.inverse ? -g.c.scale : g.c.scale, angle);
  const float inv_size = 1.0f / static_cast<float>(g.c.size);
  const int all = g.steps[0] + g.steps[1];
  const int first = static_cast<int>(static_cast<int64_t>(all) * split / g.splits);
  const int last = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / g.splits);
#pragma unroll 1
  for (int n = 0; n < 2; ++n) {
    const HeadSet& set = g.c.set[n];
    const int off = n ? g.steps[0] : 0;
    const int lo = first > off ? first - off : 0;
    const int hi = last - off < g.steps[n] ? last - off : g.steps[n];
    if (lo >= hi) continue;
    const T* x = static_cast<const T*>(set.x) + b * set.xs.batch + t * set.xs.token;
    T* y = static_cast<T*>(set.y) + b * set.ys.batch + t * set.ys.token;
    float gl[K][VE], gh[K][VE];
    if constexpr (NORM) head_gamma<VE, K>(sh.gamma[n], u, gl, gh);
    HeadRow<T, VE, K> next;
    int64_t h = static_cast<int64_t>(lo) * rows + row;
    head_load<T, VE, K>(next, x + h * set.xs.head, h < set.heads, u);
#pragma unroll 1
    for (int i = lo; i < hi; ++i, h += rows) {
      const HeadRow<T, VE, K> now = next;
      if (i + 1 < hi)
        head_load<T, VE, K>(next, x + (h + rows) * set.xs.head, h + rows < set.heads, u);
      float vl[K][VE], vh[K][VE];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unpack(now.lo[k], vl[k]);
        unpack(now.hi[k], vh[k]);
      }
      if constexpr (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            sum = fmaf(vl[k][e], vl[k][e], sum);
            sum = fmaf(vh[k][e], vh[k][e], sum);
          }
        sum = seg_sum(sum, g.lanes);
        const float r = rsqrtf(sum * inv_size + g.c.eps);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            vl[k][e] = vl[k][e] * r * gl[k][e];
            vh[k][e] = vh[k][e] * r * gh[k][e];
          }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) turn<VE>(g, u.pair[k], angle.c[k], angle.s[k], vl[k], vh[k]);
      head_store<T, VE, K>(y + h * set.ys.head, h < set.heads, u, vl, vh);
    }
  }
}

// -- gradient ---------------------------------------------------------------------

// With da = the rotation transposed of dy and g = da gamma:
//   dx = r (g - u mean(g u)),  dgamma = sum over rows of da u.
// The first parts[0] CTAs take the queries, the others the keys; each keeps its
// columns' sums in registers over all its rows and stores them as one part.
template <typename T, int VE, int K>
__global__ void __launch_bounds__(32 * kHeadWarps) heads_grad_kernel(const HeadsArgs g) {
  __shared__ HeadShared sh;
  __shared__ float red[kHeadWarps][kMaxHeadSize];
  pdl_wait();
  pdl_trigger();
  head_shared(g, sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (g.lanes - 1), row = lane / g.lanes, rows = 32 / g.lanes;
  const int n = blockIdx.x >= static_cast<unsigned>(g.parts[0]);
  const HeadSet& set = g.c.set[n];
  const unsigned part = blockIdx.x - (n ? g.parts[0] : 0);
  const HeadUnits<VE, K> u = head_units<VE, K>(g, sub);
  const float inv_size = 1.0f / static_cast<float>(g.c.size);
  float gl[K][VE], gh[K][VE];
  head_gamma<VE, K>(sh.gamma[n], u, gl, gh);
  float dl[K][VE] = {}, dh[K][VE] = {};
  const unsigned long long items = static_cast<unsigned long long>(g.tokens) * g.splits;
  const unsigned long long stride = static_cast<unsigned long long>(g.parts[n]) * kHeadWarps;
#pragma unroll 1
  for (unsigned long long item = static_cast<unsigned long long>(part) * kHeadWarps + warp;
       item < items; item += stride) {
    const unsigned token = static_cast<unsigned>(item / g.splits);
    const int split = static_cast<int>(item - static_cast<unsigned long long>(token) * g.splits);
    const unsigned b = token / g.seq, t = token - b * g.seq;
    const int first = static_cast<int>(static_cast<int64_t>(g.steps[n]) * split / g.splits);
    const int last = static_cast<int>(static_cast<int64_t>(g.steps[n]) * (split + 1) / g.splits);
    if (first >= last) continue;
    HeadAngles<VE, K> angle;
    head_angles<VE, K>(g, sh.steps, u, b, t, -g.c.scale, angle);
    const T* x = static_cast<const T*>(set.x) + b * set.xs.batch + t * set.xs.token;
    const T* dy = static_cast<const T*>(set.dy) + b * set.dys.batch + t * set.dys.token;
    T* dx = static_cast<T*>(set.y);
    if (dx) dx += b * set.ys.batch + t * set.ys.token;
    HeadRow<T, VE, K> nx, nd;
    int64_t h = static_cast<int64_t>(first) * rows + row;
    head_load<T, VE, K>(nx, x + h * set.xs.head, h < set.heads, u);
    head_load<T, VE, K>(nd, dy + h * set.dys.head, h < set.heads, u);
#pragma unroll 1
    for (int i = first; i < last; ++i, h += rows) {
      const HeadRow<T, VE, K> rx = nx, rd = nd;
      if (i + 1 < last) {
        head_load<T, VE, K>(nx, x + (h + rows) * set.xs.head, h + rows < set.heads, u);
        head_load<T, VE, K>(nd, dy + (h + rows) * set.dys.head, h + rows < set.heads, u);
      }
      float al[K][VE], ah[K][VE], xl[K][VE], xh[K][VE];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unpack(rx.lo[k], xl[k]);
        unpack(rx.hi[k], xh[k]);
        unpack(rd.lo[k], al[k]);
        unpack(rd.hi[k], ah[k]);
        turn<VE>(g, u.pair[k], angle.c[k], angle.s[k], al[k], ah[k]);
      }
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          sum = fmaf(xl[k][e], xl[k][e], sum);
          sum = fmaf(xh[k][e], xh[k][e], sum);
        }
      const float r = rsqrtf(seg_sum(sum, g.lanes) * inv_size + g.c.eps);
      float dot = 0.0f;
      // a lane without a row here has dy = 0, and x = 0: nothing is added unless r is
      // infinite (eps 0), so its sums are left alone
      const bool in = h < set.heads;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          xl[k][e] *= r;
          xh[k][e] *= r;
          if (in) {
            dl[k][e] = fmaf(al[k][e], xl[k][e], dl[k][e]);
            dh[k][e] = fmaf(ah[k][e], xh[k][e], dh[k][e]);
          }
          al[k][e] *= gl[k][e];
          ah[k][e] *= gh[k][e];
          dot = fmaf(al[k][e], xl[k][e], dot);
          dot = fmaf(ah[k][e], xh[k][e], dot);
        }
      if (!dx) continue;
      const float m = seg_sum(dot, g.lanes) * inv_size;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          al[k][e] = r * fmaf(-m, xl[k][e], al[k][e]);
          ah[k][e] = r * fmaf(-m, xh[k][e], ah[k][e]);
        }
      head_store<T, VE, K>(dx + h * set.ys.head, in, u, al, ah);
    }
  }
  if (!set.dgamma) return;
  // the groups of a warp, then the warps in order
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      for (int o = g.lanes; o < 32; o <<= 1) {
        dl[k][e] += __shfl_xor_sync(0xffffffffu, dl[k][e], o);
        dh[k][e] += __shfl_xor_sync(0xffffffffu, dh[k][e], o);
      }
      if (row == 0) {
        if (u.lo[k] >= 0) red[warp][u.lo[k] + e] = dl[k][e];
        if (u.hi[k] >= 0) red[warp][u.hi[k] + e] = dh[k][e];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < g.c.size; i += blockDim.x) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kHeadWarps; ++w) t += red[w][i];
    g.c.part[static_cast<int64_t>(blockIdx.x) * g.c.size + i] = t;
  }
}

// The parts added in a fixed order: a CTA takes 32 columns of a tensor's, its 32 warps
// every 32nd part each, then the warps' sums are added.
template <typename M>
__global__ void __launch_bounds__(1024) heads_dgamma_kernel(const float* part, M* dq, M* dk,
                                                            int size, int parts_q, int parts_k) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool keys = blockIdx.y != 0;
  M* out = keys ? dk : dq;
  if (!out) return;
  const int parts = keys ? parts_k : parts_q;
  const float* p = part + (keys ? static_cast<int64_t>(parts_q) * size : 0);
  float t = 0.0f;
  if (col < size) {
#pragma unroll 4
    for (int i = warp; i < parts; i += 32) t += p[static_cast<int64_t>(i) * size + col];
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp != 0 || col >= size) return;
  t = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) t += red[w][lane];
  out[col] = from_f32<M>(t);
}

}  // namespace b200norm
