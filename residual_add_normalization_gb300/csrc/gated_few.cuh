// gated_few.cuh -- gradients of a gated linear call of a few rows (sm_103a).
//
//   dz[r, o] = dh[r, o] * z[r, F + o] * act'(z[r, o]),  dz[r, F + o] = dh[r, o] * act(z[r, o])
//   dx = dz W,  dW = dz^T x,  db = sum of dz over the rows
//
// Bound by HBM: the weight is read and its gradient written once, element by element in the
// same place, and everything else is small.  So one launch does both: a warp has 32 * VE
// columns of the weight and walks its rows, adding dz times them to its part of dx and storing
// dz^T x; dz comes from shared memory, made by the CTA for 128 features at a time, and is not
// rounded.  A second launch adds the parts of dx.  1 x 4096 x 8192 (rows, in, out) bf16 46.6 us
// (5.8 TB/s, 86% of the copy rate; dz and two products 79), 4 x 4096 x 4096 29.8 (51), float32
// 50 (164); a row of 768 x 768 4.9 (15.2).
#pragma once

#include "launch_kernel.cuh"
#include "linear.cuh"
#include "pair.cuh"

namespace b200norm {

constexpr int kFewWarps = 8;
constexpr int kFewChunk = 128;  // features whose dz is in shared memory at a time

struct GatedFewArgs {
  const void *dh, *x, *w, *z;
  void *dw, *db;   // null: not wanted
  float* part;     // of dx, [parts][rows][in] (null: not wanted)
  int64_t rows, in, out;
  int act;
};

// R: rows at most.
template <typename T, int VE, int R>
__global__ void __launch_bounds__(32 * kFewWarps, 2) gated_few_kernel(const GatedFewArgs c) {
  pdl_wait();
  pdl_trigger();
  __shared__ alignas(16) float sdz[2][kFewChunk][R];
  __shared__ float red[kFewWarps][32 * VE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 32 * VE;
  const int64_t col = first + lane * VE;
  const bool mine = col < c.in;
  const int64_t parts = gridDim.y, part = blockIdx.y;
  const int64_t o0 = c.out * part / parts, o1 = c.out * (part + 1) / parts;
  const T* dh = static_cast<const T*>(c.dh);
  const T* z = static_cast<const T*>(c.z);
  const T* w = static_cast<const T*>(c.w) + col;
  T* dw = static_cast<T*>(c.dw) + col;
  T* db = static_cast<T*>(c.db);

  // features that a warp loads the weight of at once
  constexpr int kFewAhead = sizeof(T) * VE == 16 ? 4 : 8;
  // pairs of columns, for one instruction on both (VE 1: the second is nothing)
  constexpr int P = VE == 1 ? 1 : VE / 2;
  float2 x[R][P] = {}, acc[R][P] = {};
  auto widen = [](const Pack<T, VE>& p, float2 (&f)[P]) {
    if constexpr (VE == 1) {
      f[0] = make_float2(to_f32(p.v[0]), 0.0f);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = get2(p, i);
    }
  };
  if (c.dw && mine) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < c.rows) widen(ld_reuse<T, VE>(static_cast<const T*>(c.x) + r * c.in + col), x[r]);
  }

#pragma unroll 1
  for (int64_t base = o0; base < o1; base += kFewChunk) {
    const int n = static_cast<int>(o1 - base < kFewChunk ? o1 - base : kFewChunk);
    __syncthreads();
    with_act(c.act, [&](auto act) {
#pragma unroll 1
      for (int i = threadIdx.x; i < kFewChunk * R; i += 32 * kFewWarps) {
        const int o = i % kFewChunk, r = i / kFewChunk;
        if (o >= n) continue;
        float gate = 0.0f, up = 0.0f;
        if (r < c.rows) {
          const int64_t at = r * c.out + base + o;
          float value, slope;
          const float d = to_f32(dh[at]);
          act_both<decltype(act)::value>(to_f32(z[at + r * c.out]), value, slope);
          gate = __fmul_rn(__fmul_rn(d, to_f32(z[at + (r + 1) * c.out])), slope);
          up = __fmul_rn(d, value);
        }
        sdz[0][o][r] = gate;
        sdz[1][o][r] = up;
      }
    });
    __syncthreads();
    if (db && blockIdx.x == 0 && threadIdx.x < 2 * kFewChunk) {
      const int s = threadIdx.x / kFewChunk, o = threadIdx.x % kFewChunk;
      if (o < n) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) t += sdz[s][o][r];
        db[s * c.out + base + o] = from_f32<T>(t);
      }
    }
    if (!mine || (!c.part && !c.dw)) continue;
#pragma unroll 1
    for (int j = warp; j < n; j += kFewWarps * kFewAhead) {
      Pack<T, VE> q[kFewAhead][2] = {};
      if (c.part) {
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u) {
          const int o = j + u * kFewWarps;
          if (o >= n) continue;
#pragma unroll
          for (int s = 0; s < 2; ++s) q[u][s] = ld_stream<T, VE>(w + (s * c.out + base + o) * c.in);
        }
      }
#pragma unroll
      for (int u = 0; u < kFewAhead; ++u) {
        const int o = j + u * kFewWarps;
        if (o >= n) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float2 f[P], sum[P] = {};
          widen(q[u][s], f);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float2 d = make_float2(sdz[s][o][r], sdz[s][o][r]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
              acc[r][i] = fma2(d, f[i], acc[r][i]);
              sum[i] = fma2(d, x[r][i], sum[i]);
            }
          }
          if (!c.dw) continue;
          Pack<T, VE> out;
#pragma unroll
          for (int i = 0; i < P; ++i) {
            out.v[2 * i] = from_f32<T>(sum[i].x);
            if constexpr (VE > 1) out.v[2 * i + 1] = from_f32<T>(sum[i].y);
          }
          *reinterpret_cast<Pack<T, VE>*>(dw + (s * c.out + base + o) * c.in) = out;
        }
      }
    }
  }

  if (!c.part) return;
  // the warps' sums, added in order
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= c.rows) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      red[warp][lane * VE + 2 * i] = acc[r][i].x;
      if constexpr (VE > 1) red[warp][lane * VE + 2 * i + 1] = acc[r][i].y;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * VE; i += 32 * kFewWarps) {
      if (first + i >= c.in) continue;
      float t = 0.0f;
#pragma unroll
      for (int v = 0; v < kFewWarps; ++v) t += red[v][i];
      c.part[(part * c.rows + r) * c.in + first + i] = t;
    }
  }
}

template <typename T>
cudaError_t launch_gated_few(const GatedFewArgs& a, void* dx, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  const int parts = gated_few_parts(a.rows, a.in, a.out, sizeof(T) == 4 ? DType::F32 : DType::F16);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w) |
                        reinterpret_cast<uintptr_t>(a.dw);
  auto go = [&](auto ve, auto r) {
    constexpr int VE = decltype(ve)::value;
    const int64_t stripes = a.part || a.dw ? (a.in + 32 * VE - 1) / (32 * VE) : 1;
    return launch_pdl(gated_few_kernel<T, VE, decltype(r)::value>,
                      dim3(static_cast<unsigned>(stripes), static_cast<unsigned>(parts)),
                      32 * kFewWarps, stream, a);
  };
  // eight rows of 16-bit types: eight bytes an access, for their registers
  constexpr int kHalf = 4;
  cudaError_t e;
  if (a.rows <= 4 && a.in % kVec == 0 && all % 16 == 0) {
    e = a.rows <= 1   ? go(Const<kVec>(), Const<1>())
        : a.rows <= 2 ? go(Const<kVec>(), Const<2>())
                      : go(Const<kVec>(), Const<4>());
  } else if (a.in % kHalf == 0 && all % (kHalf * sizeof(T)) == 0) {
    e = go(Const<kHalf>(), Const<8>());
  } else {
    e = a.rows <= 2   ? go(Const<1>(), Const<2>())
        : a.rows <= 4 ? go(Const<1>(), Const<4>())
                      : go(Const<1>(), Const<8>());
  }
  if (e != cudaSuccess || !a.part) return e;
  const int64_t n = a.rows * a.in;
  return launch_pdl(linear_db_kernel<T>, dim3(static_cast<unsigned>((n + 31) / 32)), 1024, stream,
                    static_cast<const float*>(a.part), static_cast<T*>(dx), n, parts, false);
}

}  // namespace b200norm
