// linear_launch.cuh -- host-side launch, for one element type, of the linear
// operator's kernels that do not use the tensor cores.
#pragma once

#include "launch_kernel.cuh"
#include "linear.cuh"

namespace b200norm {

// Tiles of 128 x 128 from which the plain product takes them.
constexpr int64_t kPlainLargeTiles = 128;

inline bool vectors_ok(const Operand& o, int64_t es) {
  return o.ld * es % 16 == 0 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0;
}

inline PlainProduct plain_args(const Product& p) {
  const int64_t es = static_cast<int64_t>(dtype_size(p.t));
  return {p.a.p, p.b.p, p.a.ld, p.b.ld, vectors_ok(p.a, es), vectors_ok(p.b, es),
          p.M, p.N, p.K, p.epi};
}

template <int TILE>
cudaError_t launch_plain_tile(const Product& p, int splits, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.M + TILE - 1) / TILE * splits),
                  static_cast<unsigned>((p.N + TILE - 1) / TILE));
  auto* fn = !p.a.k_contiguous    ? linear_plain_kernel<TILE, false, false>
             : p.b.k_contiguous ? linear_plain_kernel<TILE, true, true>
                                : linear_plain_kernel<TILE, true, false>;
  if (PlainShape<TILE>::kSmem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(PlainShape<TILE>::kSmem));
    if (e != cudaSuccess) return e;
  }
  return launch_clusters(fn, grid, PlainShape<TILE>::kThreads, splits, PlainShape<TILE>::kSmem,
                         stream, plain_args(p));
}

// float32 products.
inline cudaError_t launch_plain(const Product& p, cudaStream_t stream) {
  // large tiles once they fill the GPU
  if ((p.M + 127) / 128 * ((p.N + 127) / 128) >= kPlainLargeTiles)
    return launch_plain_tile<128>(p, 1, stream);
  // K split while an SM has fewer than four tiles and a part eight slices
  const int64_t tiles = (p.M + 63) / 64 * ((p.N + 63) / 64);
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= 4 * 152 && p.K / (splits * 2) >= 8 * kPlainK)
    splits *= 2;
  return launch_plain_tile<64>(p, splits, stream);
}

template <typename T, int VE>
cudaError_t launch_rows_ve(const Product& p, cudaStream_t stream) {
  const PlainProduct a = plain_args(p);
  auto go = [&](auto* fn, int no) {
    const int64_t per = static_cast<int64_t>(kRowsWarps) * no;
    return launch_pdl(fn, dim3(static_cast<unsigned>((p.N + per - 1) / per)), 32 * kRowsWarps,
                      stream, a);
  };
  if (p.M <= 1) return go(linear_rows_kernel<T, VE, 1, 1, 8>, 1);
  if (p.M <= 2) return go(linear_rows_kernel<T, VE, 2, 2, 4>, 2);
  return go(linear_rows_kernel<T, VE, 4, 2, 4>, 2);
}

template <typename T>
cudaError_t launch_rows(const Product& p, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  if (p.K % VE == 0 && vectors_ok(p.a, sizeof(T)) && vectors_ok(p.b, sizeof(T)))
    return launch_rows_ve<T, VE>(p, stream);
  return launch_rows_ve<T, 1>(p, stream);
}

template <typename T>
cudaError_t launch_dz(const LinearDzCall& c, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  const int parts = c.rows > 0 ? linear_db_parts(c.rows, c.out) : 0;
  cudaError_t e = cudaSuccess;
  if (parts > 0) {
    const Operand dy{c.dy, c.out, true}, z{c.z, c.out, true}, dz{c.dz, c.ldz, true};
    const bool vec =
        vectors_ok(dy, sizeof(T)) && vectors_ok(z, sizeof(T)) && vectors_ok(dz, sizeof(T));
    const int cols = 32 * (vec ? VE : 1);
    const dim3 grid(static_cast<unsigned>((c.out + cols - 1) / cols), parts);
    e = vec ? launch_pdl(linear_dz_kernel<T, VE>, grid, 32 * kDzWarps, stream, c, parts)
            : launch_pdl(linear_dz_kernel<T, 1>, grid, 32 * kDzWarps, stream, c, parts);
  }
  if (e == cudaSuccess && c.db)
    e = launch_pdl(linear_db_kernel<T>, dim3(static_cast<unsigned>((c.out + 31) / 32)), 1024,
                   stream, static_cast<const float*>(c.part), static_cast<T*>(c.db), c.out, parts);
  return e;
}

// Dense rows of n elements to rows pitch16(n) apart, of one operand or two.
template <typename T>
cudaError_t launch_pack(const void* src0, void* dst0, int64_t rows0, const void* src1, void* dst1,
                        int64_t rows1, int64_t n, cudaStream_t stream) {
  const int64_t words = pitch16(n) / 8;
  int64_t grid = ((rows0 + rows1) * words + 255) / 256;
  if (grid > 152 * 16) grid = 152 * 16;
  const PackRows<T> a{static_cast<const T*>(src0), static_cast<T*>(dst0), rows0};
  const PackRows<T> b{static_cast<const T*>(src1), static_cast<T*>(dst1), rows1};
  return launch_pdl(linear_pack_kernel<T>, dim3(static_cast<unsigned>(grid)), 256, stream, a, b, n,
                    words);
}

}  // namespace b200norm
