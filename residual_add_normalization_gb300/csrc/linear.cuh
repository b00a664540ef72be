// linear.cuh -- device helpers of the linear operator: the activations, their
// derivatives, and the plain tiled product (sm_103a).
#pragma once

#include "common.cuh"
#include "linear.h"

namespace b200norm {

// ---------------------------------------------------------------------------
// Activations in binary32
//   SiLU       z * s(z),       s(z) = 1 / (1 + e^-z)
//   GELU       z * P(z),       P(z) = erfc(-z / sqrt 2) / 2 (no cancellation in
//                              the tail, where 1 + erf would lose every digit)
//   GELU tanh  z * s(2 w),     w = sqrt(2/pi) (z + 0.044715 z^3): the tanh form
//                              z (1 + tanh w) / 2 rewritten, again for the tail
//   ReLU       z for z > 0, else 0 (a NaN stays a NaN)
// ---------------------------------------------------------------------------
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float sigmoid_f32(float z) {
  return rcp_approx(1.0f + ex2_approx(-z * kLog2E));
}

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case kActSilu: return z * sigmoid_f32(z);
    case kActGelu: return z * (0.5f * erfcf(-z * kSqrtHalf));
    case kActGeluTanh:
      return z * sigmoid_f32(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
    case kActRelu: return z <= 0.0f ? 0.0f : z;
    default: return z;
  }
}

// The derivative.  Past the cut-offs it is 0 or 1 to the last bit of binary32,
// and the products below would meet 0 * infinity.
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActSilu: {
      if (fabsf(z) >= 104.0f) return z > 0.0f ? 1.0f : 0.0f;
      const float s = sigmoid_f32(z);
      return s * (1.0f + z * (1.0f - s));
    }
    case kActGelu: {
      if (fabsf(z) >= 16.0f) return z > 0.0f ? 1.0f : 0.0f;
      return 0.5f * erfcf(-z * kSqrtHalf) +
             z * kInvSqrt2Pi * ex2_approx(-0.5f * kLog2E * z * z);
    }
    case kActGeluTanh: {
      if (fabsf(z) >= 16.0f) return z > 0.0f ? 1.0f : 0.0f;
      const float p = sigmoid_f32(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
      return p + z * p * (1.0f - p) * kTwoSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z * z);
    }
    case kActRelu: return z > 0.0f ? 1.0f : 0.0f;
    default: return 1.0f;
  }
}

// ---------------------------------------------------------------------------
// Plain tiled product: any sizes, strides and alignment, binary32 sums.  A CTA
// of 256 threads makes a 64 x 64 tile, 4 x 4 per thread, through shared memory.
// ---------------------------------------------------------------------------
struct PlainProduct {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool a_kc, b_kc;
  int64_t M, N, K;
  Epilogue e;
};

constexpr int kPlainTile = 64;
constexpr int kPlainK = 16;

template <typename T>
__device__ __forceinline__ float plain_elem(const T* p, int64_t ld, bool kc, int64_t i, int64_t k,
                                            int64_t ni, int64_t nk) {
  if (i >= ni || k >= nk) return 0.0f;
  return to_f32(kc ? p[i * ld + k] : p[k * ld + i]);
}

template <typename T>
__global__ void __launch_bounds__(256) linear_plain_kernel(const PlainProduct p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float as[kPlainK][kPlainTile + 4], bs[kPlainK][kPlainTile + 4];
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kPlainTile;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kPlainTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += kPlainK) {
#pragma unroll
    for (int j = 0; j < kPlainTile * kPlainK / 256; ++j) {
      const int e = threadIdx.x + j * 256;
      // neighbouring threads take neighbouring elements of the contiguous index
      const int ai = p.a_kc ? e / kPlainK : e % kPlainTile;
      const int ak = p.a_kc ? e % kPlainK : e / kPlainTile;
      as[ak][ai] = plain_elem(a, p.lda, p.a_kc, m0 + ai, k0 + ak, p.M, p.K);
      const int bi = p.b_kc ? e / kPlainK : e % kPlainTile;
      const int bk = p.b_kc ? e % kPlainK : e / kPlainTile;
      bs[bk][bi] = plain_elem(b, p.ldb, p.b_kc, n0 + bi, k0 + bk, p.N, p.K);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlainK; ++k) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = as[k][ty * 4 + i];
        bv[i] = bs[k][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
  const T* bias = static_cast<const T*>(p.e.bias);
  const T* res = static_cast<const T*>(p.e.residual);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= p.N) continue;
      float z = acc[i][j];
      if (bias) z += to_f32(bias[n]);
      if (p.e.z) static_cast<T*>(p.e.z)[m * p.N + n] = from_f32<T>(z);
      float y = act_value(z, p.e.act);
      if (res) y += to_f32(res[m * p.N + n]);
      static_cast<T*>(p.e.y)[m * p.N + n] = from_f32<T>(y);
    }
  }
}

// ---------------------------------------------------------------------------
// dz = dy * act'(z), rounded to T because it is an operand of both products
// (the rounding of a tensor of type T, half a step), and its column sums, taken
// before that rounding.  CTA (stripe, part): a column per thread, rows in order.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) linear_dz_kernel(const LinearDzCall c, int parts) {
  pdl_wait();
  pdl_trigger();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= c.out) return;
  const int part = blockIdx.y;
  const int64_t r0 = c.rows * part / parts, r1 = c.rows * (part + 1) / parts;
  const T* dy = static_cast<const T*>(c.dy);
  const T* z = static_cast<const T*>(c.z);
  T* dz = static_cast<T*>(c.dz);
  float sum = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    float d = to_f32(dy[r * c.out + col]);
    if (c.act != kActNone) d *= act_slope(to_f32(z[r * c.out + col]), c.act);
    if (dz) dz[r * c.ldz + col] = from_f32<T>(d);
    sum += d;
  }
  if (c.db) c.part[part * c.out + col] = sum;
}

// The parts added in order.
template <typename T>
__global__ void __launch_bounds__(256) linear_db_kernel(const float* part, T* db, int64_t out,
                                                        int parts) {
  pdl_wait();
  pdl_trigger();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= out) return;
  float t = 0.0f;
  for (int p = 0; p < parts; ++p) t += part[p * out + col];
  db[col] = from_f32<T>(t);
}

}  // namespace b200norm
