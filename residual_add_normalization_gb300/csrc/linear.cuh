// linear.cuh -- device helpers of the linear operator: the activations, their
// derivatives, and the plain tiled product (sm_103a).
#pragma once

#include "common.cuh"
#include "linear.h"
#include "pair.cuh"

namespace b200norm {

// ---------------------------------------------------------------------------
// Activations in binary32, with s(z) = 1 / (1 + e^-z) and P the normal
// distribution function:
//   SiLU       z * s(z)
//   GELU       z * P(z)
//   GELU tanh  z * s(2 w),   w = sqrt(2/pi) (z + 0.044715 z^3): the tanh form
//              z (1 + tanh w) / 2 rewritten, so that its tail keeps its digits
//   ReLU       z for z > 0, else 0 (a NaN stays a NaN)
//
// P's tail, P(-|z|) = e^(-z^2 / 2) * Q(|z|), has no cancellation; Q (half the
// scaled complementary error function of |z| / sqrt 2) is a polynomial in
// t = 1 / (1 + 0.3 |z|) without constant term, fitted to it on [0, 14] by
// least squares reweighted towards the smallest largest relative error: 1.5e-7,
// 4.6e-7 evaluated in binary32.  The library function for the same costs more
// than twice the instructions, which the epilogue of a product with a short sum
// has no room for (16384 x 512 x 512 bf16 with GELU: 49 us, 15 without).
// ---------------------------------------------------------------------------
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float sigmoid_f32(float z) {
  return rcp_approx(1.0f + ex2_approx(-z * kLog2E));
}

// e^(-z^2 / 2) and P(z)
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  const float t = rcp_approx(fmaf(0.3f, fabsf(z), 1.0f));
  float q = 0.03567487746477127f;
  q = fmaf(q, t, -0.15720349550247192f);
  q = fmaf(q, t, 0.20635420083999634f);
  q = fmaf(q, t, -0.05368424579501152f);
  q = fmaf(q, t, 0.12856192886829376f);
  q = fmaf(q, t, 0.09991341084241867f);
  q = fmaf(q, t, 0.12075396627187729f);
  q = fmaf(q, t, 0.11962930113077164f);
  bell = ex2_approx((-0.5f * kLog2E) * z * z);
  const float tail = q * t * bell;
  return z >= 0.0f ? 1.0f - tail : tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActSilu) return z * sigmoid_f32(z);
  if constexpr (ACT == kActGelu) {
    float bell;
    return z * normal_cdf(z, bell);
  }
  if constexpr (ACT == kActGeluTanh)
    return z * sigmoid_f32(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
  if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;
  return z;
}

// The derivative.  Past the cut-offs it is 0 or 1 to the last bit of binary32,
// and the products below would meet 0 * infinity.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f32(z);
    const float d = s * (1.0f + z * (1.0f - s));
    return fabsf(z) >= 104.0f ? (z > 0.0f ? 1.0f : 0.0f) : d;
  }
  if constexpr (ACT == kActGelu) {
    float bell;
    const float p = normal_cdf(z, bell);
    const float d = fmaf(z * kInvSqrt2Pi, bell, p);
    return fabsf(z) >= 16.0f ? (z > 0.0f ? 1.0f : 0.0f) : d;
  }
  if constexpr (ACT == kActGeluTanh) {
    const float p = sigmoid_f32(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
    const float d =
        p + z * p * (1.0f - p) * kTwoSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z * z);
    return fabsf(z) >= 16.0f ? (z > 0.0f ? 1.0f : 0.0f) : d;
  }
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  return 1.0f;
}

// f(integral constant) for the activation code, so that loops over elements
// hold one activation each.
template <int N>
struct Const {
  static constexpr int value = N;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActSilu: return f(Const<kActSilu>());
    case kActGelu: return f(Const<kActGelu>());
    case kActGeluTanh: return f(Const<kActGeluTanh>());
    case kActRelu: return f(Const<kActRelu>());
    default: return f(Const<kActNone>());
  }
}

// ---------------------------------------------------------------------------
// Tiled product on the binary32 units: float32 operands, and 16-bit ones for
// which the tensor cores have nothing to do (an empty sum).  Any sizes, strides
// and alignment; binary32 sums, k in order.  A CTA makes a TILE x TILE tile, 8
// rows by 8 (TILE 128) or 4 (64) columns per thread, two products per
// instruction; operand slices of 16 of k pass through two shared-memory buffers,
// the next slice on its way from global memory meanwhile.  Bound by the binary32
// units: 8 + 8 values from shared memory feed 64 products.
//
// With few tiles the CTAs of a cluster each take a part of K (TILE 64) and add
// their sums through distributed shared memory, in rank order.
// ---------------------------------------------------------------------------
struct PlainProduct {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool a_vec, b_vec;   // rows are whole 16-byte vectors
  int64_t M, N, K;
  Epilogue e;
};

constexpr int kPlainK = 16;

template <int TILE>
struct PlainShape {
  static constexpr int kThreads = TILE == 128 ? 256 : 128;
  static constexpr int kCols = TILE == 128 ? 8 : 4;   // per thread
  static constexpr int kQuads = TILE * kPlainK / 4 / kThreads;  // of an operand, per thread
  static constexpr int kPitch = TILE + 4;
};

// One operand's slice [16][TILE] (k major) by way of registers.
template <typename T, int TILE, bool KC>
struct PlainSlice {
  using S = PlainShape<TILE>;
  float4 q[S::kQuads];

  // quad u of this thread: four of k (KC) or four of i, from (i, k) on
  __device__ __forceinline__ static void place(int u, int& i, int& k) {
    const int id = threadIdx.x + u * S::kThreads;
    if constexpr (KC) {
      i = id / (kPlainK / 4);
      k = id % (kPlainK / 4) * 4;
    } else {
      i = id % (TILE / 4) * 4;
      k = id / (TILE / 4);
    }
  }

  __device__ __forceinline__ void load(const T* p, int64_t ld, bool vec, int64_t i0, int64_t k0,
                                       int64_t ni, int64_t nk) {
#pragma unroll
    for (int u = 0; u < S::kQuads; ++u) {
      int di, dk;
      place(u, di, dk);
      const int64_t i = i0 + di, k = k0 + dk;
      const bool in = KC ? (i < ni && k + 3 < nk) : (k < nk && i + 3 < ni);
      if constexpr (sizeof(T) == 4) {
        if (vec && in) {
          q[u] = __ldg(reinterpret_cast<const float4*>(p + (KC ? i * ld + k : k * ld + i)));
          continue;
        }
      }
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t ie = KC ? i : i + e, ke = KC ? k + e : k;
        f[e] = ie < ni && ke < nk ? to_f32(p[KC ? ie * ld + ke : ke * ld + ie]) : 0.0f;
      }
      q[u] = make_float4(f[0], f[1], f[2], f[3]);
    }
  }

  __device__ __forceinline__ void put(float (*s)[S::kPitch]) const {
#pragma unroll
    for (int u = 0; u < S::kQuads; ++u) {
      int i, k;
      place(u, i, k);
      if constexpr (KC) {
        s[k][i] = q[u].x;
        s[k + 1][i] = q[u].y;
        s[k + 2][i] = q[u].z;
        s[k + 3][i] = q[u].w;
      } else {
        *reinterpret_cast<float4*>(&s[k][i]) = q[u];
      }
    }
  }
};

template <typename T, int TILE, bool A_KC, bool B_KC>
__global__ void __launch_bounds__(PlainShape<TILE>::kThreads)
linear_plain_kernel(const PlainProduct p) {
  using S = PlainShape<TILE>;
  constexpr int C = S::kCols;
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float slices_of[2][2][kPlainK][S::kPitch];
  float(*as)[kPlainK][S::kPitch] = slices_of[0];
  float(*bs)[kPlainK][S::kPitch] = slices_of[1];
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  const unsigned csize = TILE == 64 ? cluster_size() : 1u;
  const unsigned rank = csize > 1 ? cluster_rank() : 0u;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / csize) * TILE;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * TILE;
  // this CTA's part of K: whole slices
  const int64_t slices = (p.K + kPlainK - 1) / kPlainK;
  const int64_t k_lo = slices * rank / csize * kPlainK;
  int64_t k_hi = slices * (rank + 1) / csize * kPlainK;
  if (k_hi > p.K) k_hi = p.K;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // rows ty * 4 + {0..3} of both halves of the tile (TILE 64: of 32 rows each);
  // columns tx * 4 + {0..3}, of both halves with eight
  constexpr int kHalf = TILE / 2;
  float2 acc[8][C / 2] = {};
  PlainSlice<T, TILE, A_KC> qa;
  PlainSlice<T, TILE, B_KC> qb;
  qa.load(a, p.lda, p.a_vec, m0, k_lo, p.M, k_hi);
  qb.load(b, p.ldb, p.b_vec, n0, k_lo, p.N, k_hi);
  int buf = 0;
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += kPlainK, buf ^= 1) {
    qa.put(as[buf]);
    qb.put(bs[buf]);
    __syncthreads();  // and everyone has left the other buffer
    if (k0 + kPlainK < k_hi) {
      qa.load(a, p.lda, p.a_vec, m0, k0 + kPlainK, p.M, k_hi);
      qb.load(b, p.ldb, p.b_vec, n0, k0 + kPlainK, p.N, k_hi);
    }
#pragma unroll
    for (int k = 0; k < kPlainK; ++k) {
      float av[8];
      float2 bv[C / 2];
      *reinterpret_cast<float4*>(av) = *reinterpret_cast<const float4*>(&as[buf][k][ty * 4]);
      *reinterpret_cast<float4*>(av + 4) =
          *reinterpret_cast<const float4*>(&as[buf][k][kHalf + ty * 4]);
#pragma unroll
      for (int h = 0; h < C / 4; ++h) {
        const float4 t = *reinterpret_cast<const float4*>(&bs[buf][k][h * kHalf + tx * 4]);
        bv[2 * h] = make_float2(t.x, t.y);
        bv[2 * h + 1] = make_float2(t.z, t.w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < C / 2; ++j) acc[i][j] = fma2(both(av[i]), bv[j], acc[i][j]);
    }
  }
  const T* bias = static_cast<const T*>(p.e.bias);
  const T* res = static_cast<const T*>(p.e.residual);
  // (the gradients' products are stored as they are)
  constexpr bool kFull = A_KC && B_KC;
  auto before = [&](int64_t m, int64_t n, float z) {  // z of (m, n), from its sum
    if constexpr (kFull) {
      if (m >= p.M || n >= p.N) return z;
      if (bias) z += to_f32(bias[n]);
      if (p.e.z) static_cast<T*>(p.e.z)[m * p.N + n] = from_f32<T>(z);
    }
    return z;
  };
  auto after = [&](int64_t m, int64_t n, float y) {
    if (m >= p.M || n >= p.N) return;
    if constexpr (kFull) {
      if (res) y += to_f32(res[m * p.N + n]);
    }
    static_cast<T*>(p.e.y)[m * p.N + n] = from_f32<T>(y);
  };
  if constexpr (TILE == 64) {
    if (csize > 1) {
      static_assert(sizeof(slices_of) >= 64 * 64 * 4, "a tile's sums fit the slices' memory");
      float* sums = &slices_of[0][0][0][0];  // [64][64]
      __syncthreads();  // the slices have been read
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(sums + ((i / 4) * kHalf + ty * 4 + i % 4) * 64 + tx * 4) =
            make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
      cluster_sync();
      const int per = 64 * 16 / static_cast<int>(csize);  // quads of this rank
      for (int q = threadIdx.x; q < per; q += S::kThreads) {
        const int at = static_cast<int>(rank) * per + q;
        float t[4] = {};
        for (unsigned c = 0; c < csize; ++c) {
          const float4 v = ld_cluster_f32x4(reinterpret_cast<const float4*>(sums) + at, c);
          t[0] += v.x;
          t[1] += v.y;
          t[2] += v.z;
          t[3] += v.w;
        }
        const int64_t m = m0 + at / 16, n = n0 + at % 16 * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = before(m, n + e, t[e]);
        if constexpr (kFull)
          with_act(p.e.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = act_value<decltype(act)::value>(t[e]);
          });
#pragma unroll
        for (int e = 0; e < 4; ++e) after(m, n + e, t[e]);
      }
      cluster_sync();  // the peers may still read this CTA's sums
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = m0 + (i / 4) * kHalf + ty * 4 + i % 4;
    float t[C];
#pragma unroll
    for (int j = 0; j < C; ++j)
      t[j] = before(m, n0 + (j / 4) * kHalf + tx * 4 + j % 4,
                    j % 2 ? acc[i][j / 2].y : acc[i][j / 2].x);
    if constexpr (kFull)
      with_act(p.e.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < C; ++j) t[j] = act_value<decltype(act)::value>(t[j]);
      });
#pragma unroll
    for (int j = 0; j < C; ++j) after(m, n0 + (j / 4) * kHalf + tx * 4 + j % 4, t[j]);
  }
}

// ---------------------------------------------------------------------------
// Few rows of x (at most R): bound by reading the weight once.  A warp takes NO
// columns of the result; its lanes share the sum, U vectors of each weight row on
// their way at once, and the rows of x come from L1.  The binary32 sums of the
// lanes are added by butterflies.
// ---------------------------------------------------------------------------
constexpr int kRowsWarps = 8;

template <typename T, int VE, int R, int NO, int U>
__global__ void __launch_bounds__(32 * kRowsWarps) linear_rows_kernel(const PlainProduct p) {
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(p.a);
  const T* w = static_cast<const T*>(p.b);
  const int lane = threadIdx.x & 31;
  const int64_t n0 =
      (static_cast<int64_t>(blockIdx.x) * kRowsWarps + (threadIdx.x >> 5)) * NO;
  if (n0 >= p.N) return;
  const int nvec = static_cast<int>(p.K / VE);
  const T* row[NO];
#pragma unroll
  for (int o = 0; o < NO; ++o) row[o] = w + (n0 + o < p.N ? n0 + o : p.N - 1) * p.ldb;
  // even and odd elements apart, two products per instruction
  float2 acc[R][NO] = {};
  for (int v0 = lane; v0 < nvec; v0 += 32 * U) {
    Pack<T, VE> q[U][NO];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 32 * u;
      if (v >= nvec) continue;
#pragma unroll
      for (int o = 0; o < NO; ++o) q[u][o] = ld_reuse<T, VE>(row[o] + static_cast<int64_t>(v) * VE);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 32 * u;
      if (v >= nvec) continue;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= p.M) continue;
        const Pack<T, VE> xv = ld_reuse<T, VE>(x + r * p.lda + static_cast<int64_t>(v) * VE);
#pragma unroll
        for (int o = 0; o < NO; ++o) {
          if constexpr (VE == 1) {
            acc[r][o].x = fmaf(to_f32(xv.v[0]), to_f32(q[u][o].v[0]), acc[r][o].x);
          } else {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) acc[r][o] = fma2(get2(xv, i), get2(q[u][o], i), acc[r][o]);
          }
        }
      }
    }
  }
  // lane (r, o) keeps that sum
  float mine = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int o = 0; o < NO; ++o) {
      const float t = warp_sum(acc[r][o].x + acc[r][o].y);
      if (lane == r * NO + o) mine = t;
    }
  const int r = lane / NO;
  const int64_t n = n0 + lane % NO;
  if (r >= R || r >= p.M || n >= p.N) return;
  const int64_t at = r * p.N + n;
  const T* bias = static_cast<const T*>(p.e.bias);
  const T* res = static_cast<const T*>(p.e.residual);
  float z = mine;
  if (bias) z += to_f32(bias[n]);
  if (p.e.z) static_cast<T*>(p.e.z)[at] = from_f32<T>(z);
  float y = 0.0f;
  with_act(p.e.act, [&](auto act) { y = act_value<decltype(act)::value>(z); });
  if (res) y += to_f32(res[at]);
  static_cast<T*>(p.e.y)[at] = from_f32<T>(y);
}

// ---------------------------------------------------------------------------
// dz = dy * act'(z), rounded to T because it is an operand of both products
// (the rounding of a tensor of type T, half a step), and its column sums, taken
// before that rounding.  Bound by HBM: two reads and a write per element.  CTA
// (stripe, part): 32 lanes by VE columns, a row per warp at a time, rows in order
// per warp; the warps' sums are added in order through shared memory.
// ---------------------------------------------------------------------------
constexpr int kDzWarps = 8;

template <typename T, int VE, int ACT>
__device__ __forceinline__ void linear_dz_rows(const LinearDzCall& c, int64_t r0, int64_t r1,
                                               int64_t col, float (&sum)[VE]) {
  const T* dy = static_cast<const T*>(c.dy);
  const T* z = static_cast<const T*>(c.z);
  T* dz = static_cast<T*>(c.dz);
  constexpr int U = 4;  // rows on their way at once
  for (int64_t r = r0; r < r1; r += U * kDzWarps) {
    Pack<T, VE> d[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r + u * kDzWarps;
      if (row >= r1) continue;
      d[u] = ld_stream<T, VE>(dy + row * c.out + col);
      if constexpr (ACT != kActNone) q[u] = ld_stream<T, VE>(z + row * c.out + col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r + u * kDzWarps;
      if (row >= r1) continue;
      float f[VE];
      unpack(d[u], f);
      if constexpr (ACT != kActNone) {
        float zf[VE];
        unpack(q[u], zf);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = __fmul_rn(f[e], act_slope<ACT>(zf[e]));
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) sum[e] = __fadd_rn(sum[e], f[e]);  // same bits without dz
      if (dz) *reinterpret_cast<Pack<T, VE>*>(dz + row * c.ldz + col) = pack_from<T, VE>(f);
    }
  }
}

template <typename T, int VE>
__global__ void __launch_bounds__(32 * kDzWarps) linear_dz_kernel(const LinearDzCall c, int parts) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[kDzWarps][32 * VE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * VE;
  const int part = blockIdx.y;
  const int64_t r0 = c.rows * part / parts, r1 = c.rows * (part + 1) / parts;
  float sum[VE] = {};
  if (col < c.out)
    with_act(c.act, [&](auto act) {
      linear_dz_rows<T, VE, decltype(act)::value>(c, r0 + warp, r1, col, sum);
    });
  if (!c.db) return;
#pragma unroll
  for (int e = 0; e < VE; ++e) red[warp][lane * VE + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VE; i += 32 * kDzWarps) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 * VE + i;
    if (at >= c.out) continue;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kDzWarps; ++w) t += red[w][i];
    c.part[part * c.out + at] = t;
  }
}

// The parts added in a fixed order: a CTA takes 32 columns, its 32 warps every
// 32nd part each, then the warps' sums are added.
template <typename T>
__global__ void __launch_bounds__(1024) linear_db_kernel(const float* part, T* db, int64_t out,
                                                         int parts) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (col < out) {
#pragma unroll 4
    for (int p = warp; p < parts; p += 32) t += part[p * out + col];
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp != 0 || col >= out) return;
  t = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) t += red[w][lane];
  db[col] = from_f32<T>(t);
}

// ---------------------------------------------------------------------------
// An operand whose rows do not start on 16-byte boundaries, copied to rows that
// do (tensor copies need them); `words` 16-byte words per row.  A word comes
// from the two aligned words that hold it, or, at the tensor's ends, from its
// elements.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) linear_pack_kernel(const T* src, T* dst, int64_t rows,
                                                          int64_t n, int64_t words) {
  static_assert(sizeof(T) == 2, "16-bit elements");
  pdl_wait();
  pdl_trigger();
  const uintptr_t end = reinterpret_cast<uintptr_t>(src + rows * n);
  const int64_t total = rows * words;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / words, k = (i - row * words) * 8;
    const T* p = src + row * n + k;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), lo = a & ~uintptr_t{15};
    uint4 out;
    if (lo >= reinterpret_cast<uintptr_t>(src) && lo + 32 <= end) {
      const uint4* q = reinterpret_cast<const uint4*>(lo);
      const uint4 x = __ldg(q), y = __ldg(q + 1);
      const unsigned w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const int skip = static_cast<int>(a & 15) / 4, bits = static_cast<int>(a & 2) * 8;
      unsigned r[5];
#pragma unroll
      for (int j = 0; j < 5; ++j) {
        const unsigned v01 = skip & 1 ? w[j + 1 < 8 ? j + 1 : 7] : w[j];
        const unsigned v23 = skip & 1 ? w[j + 3 < 8 ? j + 3 : 7] : w[j + 2 < 8 ? j + 2 : 7];
        r[j] = skip & 2 ? v23 : v01;
      }
      out = make_uint4(__funnelshift_r(r[0], r[1], bits), __funnelshift_r(r[1], r[2], bits),
                       __funnelshift_r(r[2], r[3], bits), __funnelshift_r(r[3], r[4], bits));
    } else {
      Pack<T, 8> v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] = k + e < n ? p[e] : from_f32<T>(0.0f);
      memcpy(&out, &v, sizeof(out));
    }
    reinterpret_cast<uint4*>(dst)[i] = out;
  }
}

}  // namespace b200norm
