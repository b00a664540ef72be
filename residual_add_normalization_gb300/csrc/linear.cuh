// linear.cuh -- device helpers of the linear operator: the activations, their
// derivatives, and the plain tiled product (sm_103a).
#pragma once

#include "bulk.cuh"
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
// least squares reweighted towards the smallest largest relative error: 1.8e-7,
// about 5e-7 evaluated in binary32.  The library function for the same costs more
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

// p = s(a) and q = 1 - p, neither by a subtraction: the derivatives multiply the
// smaller one by up to 35, and 1 - p keeps no more digits of it than 1 has (33 half
// steps of the GELU tanh form's slope at z = 4.96, 2 this way).
__device__ __forceinline__ void sigmoid_pair(float a, float& p, float& q) {
  const float e = ex2_approx(-fabsf(a) * kLog2E);
  const float r = rcp_approx(1.0f + e), er = e * r;
  p = a >= 0.0f ? r : er;
  q = a >= 0.0f ? er : r;
}

// The derivative.  Past the cut-offs it is 0 or 1 to the last bit of binary32,
// and the products below would meet 0 * infinity.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActSilu) {
    float p, q;
    sigmoid_pair(z, p, q);
    const float d = p + z * p * q;
    return fabsf(z) >= 104.0f ? (z > 0.0f ? 1.0f : 0.0f) : d;
  }
  if constexpr (ACT == kActGelu) {
    float bell;
    const float p = normal_cdf(z, bell);
    const float d = fmaf(z * kInvSqrt2Pi, bell, p);
    return fabsf(z) >= 16.0f ? (z > 0.0f ? 1.0f : 0.0f) : d;
  }
  if constexpr (ACT == kActGeluTanh) {
    float p, q;
    sigmoid_pair(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z), p, q);
    const float d = p + z * p * q * kTwoSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z * z);
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
// float32 product on the binary32 units.  Any sizes, strides and alignment;
// binary32 sums, k in order.  A CTA makes a TILE x TILE tile, 8 rows by 8 (TILE
// 128) or 4 (64) columns per thread, two products per instruction.  Slices of 16
// of k are copied asynchronously into a ring of shared memory, k by i whatever
// the operand's order: 16 bytes at a time where i is contiguous and aligned, else
// by elements.  Bound by the binary32 units: 16 values from shared memory feed 64
// products.  4096^3 takes 2635 us (52 of the units' 74 TFLOP/s; the library's product
// 2302), 3000 x 1027 x 2050 307 (244).  (Pairs along k, which need no value twice,
// take 254 registers for their sums and lost a third of the rate: 4096^3 3069 us.)
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

// A sum split over the CTAs of a cluster is read from all of them at once: a read
// of a peer's shared memory takes as long as one from L2, and one after another
// eight ranks' took most of a small product's time (64 x 4096 x 4096 bf16 12.5 us).
constexpr int kMaxSplits = 8;

__device__ __forceinline__ unsigned peer_addr(const void* p, unsigned rank) {
  unsigned remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  return remote;
}
__device__ __forceinline__ float peer_load(unsigned addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(unsigned addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

constexpr int kPlainK = 16;
constexpr int kPlainStages = 4;  // 3 lose 4 percent; 6 as well, by fewer CTAs per SM
template <int TILE>
struct PlainShape {
  static constexpr int kThreads = TILE == 128 ? 256 : 128;
  static constexpr int kCols = TILE == 128 ? 8 : 4;  // per thread
  static constexpr int kPitch = TILE + 4;
  static constexpr int kStage = 2 * kPlainK * kPitch;  // floats
  static constexpr size_t kSmem = static_cast<size_t>(kPlainStages) * kStage * 4;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(float* dst, const float* src, int valid) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_addr(dst)), "l"(src), "r"(valid) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(smem_addr(dst)), "l"(src), "r"(valid) : "memory");
}

// An operand's slice from (i0, k0) on to s[kPlainK][kPitch]; zero past ni and nk.
template <int TILE, bool KC>
__device__ __forceinline__ void plain_slice(float* s, const float* p, int64_t ld, bool vec,
                                            int64_t i0, int64_t k0, int64_t ni, int64_t nk) {
  constexpr int kThreads = PlainShape<TILE>::kThreads, kPitch = PlainShape<TILE>::kPitch;
  if (!KC && vec) {
#pragma unroll
    for (int u = 0; u < TILE * kPlainK / 4 / kThreads; ++u) {
      const int id = threadIdx.x + u * kThreads, i = id % (TILE / 4) * 4, k = id / (TILE / 4);
      const bool in = i0 + i < ni && k0 + k < nk;  // ni is whole vectors
      copy_async<16>(s + k * kPitch + i, in ? p + (k0 + k) * ld + i0 + i : p, in ? 16 : 0);
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < TILE * kPlainK / kThreads; ++u) {
    const int id = threadIdx.x + u * kThreads;
    const int i = KC ? id / kPlainK : id % TILE, k = KC ? id % kPlainK : id / TILE;
    const bool in = i0 + i < ni && k0 + k < nk;
    copy_async<4>(s + k * kPitch + i,
                  in ? p + (KC ? (i0 + i) * ld + k0 + k : (k0 + k) * ld + i0 + i) : p, in ? 4 : 0);
  }
}

// (Registers: left to itself the compiler packs the small tile into 96 and loses a
// sixth; three CTAs per SM, four for the weight's gradient, measured best.  Two of
// the large tile cost a few spilled registers and gain a twentieth.)
template <int TILE, bool A_KC, bool B_KC>
__global__ void __launch_bounds__(PlainShape<TILE>::kThreads, TILE == 128 ? 2 : A_KC ? 3 : 4)
linear_plain_kernel(const PlainProduct p) {
  using S = PlainShape<TILE>;
  constexpr int C = S::kCols, kHalf = TILE / 2;
  extern __shared__ __align__(16) float ring[];
  pdl_wait();
  pdl_trigger();
  const float* a = static_cast<const float*>(p.a);
  const float* b = static_cast<const float*>(p.b);
  const unsigned csize = TILE == 64 ? cluster_size() : 1u;
  const unsigned rank = csize > 1 ? cluster_rank() : 0u;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / csize) * TILE;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * TILE;
  // this CTA's part of K: whole slices
  const int64_t slices = (p.K + kPlainK - 1) / kPlainK;
  const int64_t first = slices * rank / csize, count = slices * (rank + 1) / csize - first;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

  auto fetch = [&](int64_t t) {  // slice `first + t` into its stage (nothing past the last)
    if (t < count) {
      float* st = ring + t % kPlainStages * S::kStage;
      const int64_t k0 = (first + t) * kPlainK;
      plain_slice<TILE, A_KC>(st, a, p.lda, p.a_vec, m0, k0, p.M, p.K);
      plain_slice<TILE, B_KC>(st + kPlainK * S::kPitch, b, p.ldb, p.b_vec, n0, k0, p.N, p.K);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int t = 0; t < kPlainStages - 1; ++t) fetch(t);
  // rows ty * 4 + {0..3} and columns tx * 4 + {0..3} of a half of the tile, of
  // both halves with eight
  float2 acc[8][C / 2] = {};
  for (int64_t t = 0; t < count; ++t) {
    asm volatile("cp.async.wait_group %0;" :: "n"(kPlainStages - 2) : "memory");
    __syncthreads();  // the slice is there for all, and the one before has been read by all
    fetch(t + kPlainStages - 1);
    const float* as = ring + t % kPlainStages * S::kStage + ty * 4;
    const float* bs = ring + t % kPlainStages * S::kStage + kPlainK * S::kPitch + tx * 4;
#pragma unroll
    for (int k = 0; k < kPlainK; ++k) {
      float av[8];
      float2 bv[C / 2];
      *reinterpret_cast<float4*>(av) = *reinterpret_cast<const float4*>(as + k * S::kPitch);
      *reinterpret_cast<float4*>(av + 4) =
          *reinterpret_cast<const float4*>(as + k * S::kPitch + kHalf);
#pragma unroll
      for (int h = 0; h < C / 4; ++h) {
        const float4 v = *reinterpret_cast<const float4*>(bs + k * S::kPitch + h * kHalf);
        bv[2 * h] = make_float2(v.x, v.y);
        bv[2 * h + 1] = make_float2(v.z, v.w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < C / 2; ++j) acc[i][j] = fma2(both(av[i]), bv[j], acc[i][j]);
    }
  }
  const float* bias = static_cast<const float*>(p.e.bias);
  const float* res = static_cast<const float*>(p.e.residual);
  float* zs = static_cast<float*>(p.e.z);
  float* ys = static_cast<float*>(p.e.y);
  // four columns n.. of row m, from their sums (the gradients' products are stored
  // as they are)
  auto finish = [&](float(&t)[4], int64_t m, int64_t n) {
    constexpr int N = 4;
    if (m >= p.M) return;
    if constexpr (A_KC && B_KC) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int64_t c = n + j;
        if (c >= p.N) continue;
        if (bias) t[j] += bias[c];
        if (zs) zs[m * p.N + c] = t[j];
      }
      with_act(p.e.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = act_value<decltype(act)::value>(t[j]);
      });
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t c = n + j;
      if (c >= p.N) continue;
      if constexpr (A_KC && B_KC) {
        if (res) t[j] += res[m * p.N + c];
      }
      ys[m * p.N + c] = t[j];
    }
  };
  if constexpr (TILE == 64) {
    if (csize > 1) {
      float* sums = ring;  // [64][64]
      asm volatile("cp.async.wait_group 0;" ::: "memory");
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
#pragma unroll
        for (unsigned c0 = 0; c0 < kMaxSplits; c0 += 4) {
          float4 v[4];
#pragma unroll
          for (unsigned c = 0; c < 4; ++c)
            if (c0 + c < csize) v[c] = peer_load4(peer_addr(sums + at * 4, c0 + c));
#pragma unroll
          for (unsigned c = 0; c < 4; ++c) {
            if (c0 + c >= csize) continue;
            t[0] += v[c].x;
            t[1] += v[c].y;
            t[2] += v[c].z;
            t[3] += v[c].w;
          }
        }
        finish(t, m0 + at / 16, n0 + at % 16 * 4);
      }
      cluster_sync();  // the peers may still read this CTA's sums
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int h = 0; h < C / 4; ++h) {
      float t[4] = {acc[i][2 * h].x, acc[i][2 * h].y, acc[i][2 * h + 1].x, acc[i][2 * h + 1].y};
      finish(t, m0 + (i / 4) * kHalf + ty * 4 + i % 4, n0 + h * kHalf + tx * 4);
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
// Two operands in one launch (the second may have no rows).
template <typename T>
struct PackRows {
  const T* src;
  T* dst;
  int64_t rows;
};

template <typename T>
__global__ void __launch_bounds__(256) linear_pack_kernel(const PackRows<T> first,
                                                          const PackRows<T> second, int64_t n,
                                                          int64_t words) {
  static_assert(sizeof(T) == 2, "16-bit elements");
  pdl_wait();
  pdl_trigger();
  const int64_t total = (first.rows + second.rows) * words;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    int64_t row = i / words;
    const int64_t k = (i - row * words) * 8;
    const bool one = row < first.rows;
    if (!one) row -= first.rows;
    const T* src = one ? first.src : second.src;
    const uintptr_t end =
        reinterpret_cast<uintptr_t>(src + (one ? first.rows : second.rows) * n);
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
    reinterpret_cast<uint4*>(one ? first.dst : second.dst)[row * words + k / 8] = out;
  }
}

}  // namespace b200norm
