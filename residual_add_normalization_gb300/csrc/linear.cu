// The linear operator's host side: which kernel a product takes, and its launch.
#include "layer_launch.cuh"
#include "linear.cuh"

namespace b200norm {

namespace {

// Tiles of 128 x 128 from which the plain product takes them.
constexpr int64_t kPlainLargeTiles = 128;

size_t round_256(size_t n) { return (n + 255) / 256 * 256; }

bool vectors_ok(const Operand& o, int64_t es) {
  return o.ld * es % 16 == 0 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0;
}

PlainProduct plain_args(const Product& p) {
  const int64_t es = static_cast<int64_t>(dtype_size(p.t));
  return {p.a.p, p.b.p, p.a.ld, p.b.ld, vectors_ok(p.a, es), vectors_ok(p.b, es),
          p.M, p.N, p.K, p.epi};
}

template <typename T, int TILE>
cudaError_t launch_plain_tile(const Product& p, int splits, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.M + TILE - 1) / TILE * splits),
                  static_cast<unsigned>((p.N + TILE - 1) / TILE));
  auto* fn = !p.a.k_contiguous    ? linear_plain_kernel<T, TILE, false, false>
             : p.b.k_contiguous ? linear_plain_kernel<T, TILE, true, true>
                                : linear_plain_kernel<T, TILE, true, false>;
  return launch_clusters(fn, grid, PlainShape<TILE>::kThreads, splits, 0, stream, plain_args(p));
}

template <typename T>
cudaError_t launch_plain(const Product& p, cudaStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    // large tiles once they fill the GPU
    if ((p.M + 127) / 128 * ((p.N + 127) / 128) >= kPlainLargeTiles)
      return launch_plain_tile<T, 128>(p, 1, stream);
  }
  // K split while an SM has fewer than four tiles and a part eight slices
  const int64_t tiles = (p.M + 63) / 64 * ((p.N + 63) / 64);
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= 4 * 152 && p.K / (splits * 2) >= 8 * kPlainK)
    splits *= 2;
  return launch_plain_tile<T, 64>(p, splits, stream);
}

template <typename T, int VE>
cudaError_t launch_rows_ve(const Product& p, cudaStream_t stream) {
  const PlainProduct a = plain_args(p);
  auto go = [&](auto* fn, int no) {
    const int64_t per = static_cast<int64_t>(kRowsWarps) * no;
    return launch_pdl(fn, dim3(static_cast<unsigned>((p.N + per - 1) / per),
                               static_cast<unsigned>((p.M + 7) / 8)),
                      32 * kRowsWarps, stream, a);
  };
  if (p.M <= 1) return go(linear_rows_kernel<T, VE, 1, 1, 8>, 1);
  if (p.M <= 2) return go(linear_rows_kernel<T, VE, 2, 2, 4>, 2);
  if (p.M <= 4) return go(linear_rows_kernel<T, VE, 4, 2, 4>, 2);
  return go(linear_rows_kernel<T, VE, 8, 2, 4>, 2);
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

template <typename T>
cudaError_t launch_pack_t(const void* src, void* dst, int64_t rows, int64_t n,
                          cudaStream_t stream) {
  const int64_t words = pitch16(n) / 8;
  int64_t grid = (rows * words + 255) / 256;
  if (grid > 152 * 16) grid = 152 * 16;
  return launch_pdl(linear_pack_kernel<T>, dim3(static_cast<unsigned>(grid)), 256, stream,
                    static_cast<const T*>(src), static_cast<T*>(dst), rows, n, words);
}

// (n, k)-shaped dense rows of src to rows pitch16(n) apart at dst.
cudaError_t launch_pack(DType t, const void* src, void* dst, int64_t rows, int64_t n,
                        cudaStream_t stream) {
  return t == DType::F16 ? launch_pack_t<__half>(src, dst, rows, n, stream)
                         : launch_pack_t<__nv_bfloat16>(src, dst, rows, n, stream);
}

}  // namespace

cudaError_t launch_product(const Product& p, cudaStream_t stream) {
  const bool mma = mma_operand_ok(p.a, p.t) && mma_operand_ok(p.b, p.t) && p.K > 0;
  const bool few = mma ? p.M <= kFewRows && p.N * p.K <= kFewWeights && !p.forced.cg
                       : p.M <= (p.t == DType::F32 ? kFewRowsF32 : kFewRowsScalar);
  if (p.a.k_contiguous && p.b.k_contiguous && few) {
    switch (p.t) {
      case DType::F32: return launch_rows<float>(p, stream);
      case DType::F16: return launch_rows<__half>(p, stream);
      default: return launch_rows<__nv_bfloat16>(p, stream);
    }
  }
  if (mma) return launch_mma(p, stream);
  switch (p.t) {
    case DType::F32: return launch_plain<float>(p, stream);
    case DType::F16: return launch_plain<__half>(p, stream);
    default: return launch_plain<__nv_bfloat16>(p, stream);
  }
}

cudaError_t launch_linear_dz(const LinearDzCall& c, cudaStream_t stream) {
  switch (c.t) {
    case DType::F32: return launch_dz<float>(c, stream);
    case DType::F16: return launch_dz<__half>(c, stream);
    default: return launch_dz<__nv_bfloat16>(c, stream);
  }
}

LinearPlan linear_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16) {
  LinearPlan p = {};
  p.pack = t != DType::F32 && (in % 8 != 0 || !aligned16) && rows > kFewRowsScalar;
  if (p.pack) {
    p.w = round_256(static_cast<size_t>(rows) * pitch16(in) * 2);
    p.bytes = p.w + round_256(static_cast<size_t>(out) * pitch16(in) * 2);
  }
  return p;
}

LinearGradPlan linear_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, int act,
                                bool aligned16) {
  LinearGradPlan p = {};
  const bool half = t != DType::F32;
  p.make_dz = act != kActNone || (half && (out % 8 != 0 || !aligned16));
  p.pack = half && (in % 8 != 0 || !aligned16);
  p.ldz = half ? pitch16(out) : out;
  const size_t dz = p.make_dz ? static_cast<size_t>(rows) * p.ldz * dtype_size(t) : 0;
  p.part = round_256(dz);
  p.x = p.part + round_256(static_cast<size_t>(linear_db_parts(rows, out)) * out * 4);
  p.w = p.x + (p.pack ? round_256(static_cast<size_t>(rows) * pitch16(in) * 2) : 0);
  p.bytes = p.w + (p.pack ? round_256(static_cast<size_t>(out) * pitch16(in) * 2) : 0);
  return p;
}

cudaError_t launch_linear(const LinearCall& c, const LinearPlan& plan, cudaStream_t stream) {
  Operand x{c.x, c.in, true}, w{c.w, c.in, true};
  if (plan.pack) {
    char* ws = static_cast<char*>(c.workspace);
    cudaError_t e = launch_pack(c.t, c.x, ws + plan.x, c.rows, c.in, stream);
    if (e == cudaSuccess) e = launch_pack(c.t, c.w, ws + plan.w, c.out, c.in, stream);
    if (e != cudaSuccess) return e;
    x = {ws + plan.x, pitch16(c.in), true};
    w = {ws + plan.w, pitch16(c.in), true};
  }
  const Product p{x, w, c.rows, c.out, c.in, {c.bias, c.residual, c.y, c.z, c.act}, c.t, c.forced};
  return launch_product(p, stream);
}

cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream) {
  char* ws = static_cast<char*>(c.workspace);
  void* made = plan.make_dz && (c.dx || c.dw) ? ws + plan.dz : nullptr;
  cudaError_t e = cudaSuccess;
  if (made || c.db) {
    const LinearDzCall d{c.dy, c.z, made, plan.ldz, c.db, reinterpret_cast<float*>(ws + plan.part),
                         c.rows, c.out, c.act, c.t};
    e = launch_linear_dz(d, stream);
    if (e != cudaSuccess) return e;
  }
  const void* dz = plan.make_dz ? made : c.dy;
  const int64_t ldz = plan.make_dz ? plan.ldz : c.out;
  if (c.dx && c.rows > 0) {
    Operand w{c.w, c.in, false};
    if (plan.pack) {
      e = launch_pack(c.t, c.w, ws + plan.w, c.out, c.in, stream);
      if (e != cudaSuccess) return e;
      w = {ws + plan.w, pitch16(c.in), false};
    }
    const Product p{{dz, ldz, true}, w, c.rows, c.in, c.out,
                    {nullptr, nullptr, c.dx, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
    if (e != cudaSuccess) return e;
  }
  if (c.dw) {
    Operand x{c.x, c.in, false};
    if (plan.pack && c.rows > 0) {
      e = launch_pack(c.t, c.x, ws + plan.x, c.rows, c.in, stream);
      if (e != cudaSuccess) return e;
      x = {ws + plan.x, pitch16(c.in), false};
    }
    const Product p{{dz, ldz, false}, x, c.out, c.in, c.rows,
                    {nullptr, nullptr, c.dw, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
  }
  return e;
}

}  // namespace b200norm
